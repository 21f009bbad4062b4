"""Plain 64-bit forms of the operators around the grouped product, for the tests: numpy, one
definition after the other, no code shared with the library.

Tolerances.  u = 2^-24 is fp32's unit roundoff, and `rounding` half the spacing of an output
type at a value: what one rounding to nearest may move it.  A CTA's sum of n fp32 terms is a chain of at most 32 additions per thread
(four vectors of eight), five in a warp and five across warps: 42 u relative to the sum of
magnitudes.
"""
import numpy as np
import torch

U = 2.0 ** -24
E4M3_MAX = 448.0
TINY = 2.0 ** -80
BLOCK = 128


def np64(t):
    """A tensor's values in float64 (codes given as uint8 or float8 are decoded)."""
    if t.dtype == torch.uint8:
        t = t.view(torch.float8_e4m3fn)
    if t.dtype == torch.float64 or not t.dtype.is_floating_point:
        return t.detach().cpu().numpy()
    return t.detach().cpu().to(torch.float32).numpy().astype(np.float64)


def rounding(dtype, v):
    """Half the spacing of the type's numbers at |v|: 8, 11 or 24 significant bits, subnormals
    below the smallest exponent."""
    bits, least = {torch.bfloat16: (8, -126), torch.float16: (11, -14),
                   torch.float32: (24, -126)}[dtype]
    mantissa, exponent = np.frexp(np.abs(v))      # |v| = mantissa * 2^exponent, in [0.5, 1)
    exponent = np.maximum(np.where(mantissa > 0, exponent - 1, least), least)
    return np.exp2(exponent - bits)


def close(got, want, tol, what):
    """|got - want| <= tol element by element; NaN and infinities at the same places."""
    got, want = np64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert got.shape == want.shape, f"{what}: shape {got.shape}, expected {want.shape}"
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN positions differ"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = np.isfinite(want)
    err, tol = np.abs(got - want)[fine], np.broadcast_to(tol, want.shape)[fine]
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, by up to " \
        f"{np.max(err[bad] / np.maximum(tol[bad], 1e-300)):.3g} of the tolerance"


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))),
                    np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def quantize(v, block):
    """(v / scale before its rounding, scale) per block of columns."""
    b = v.reshape(v.shape[0], -1, block)
    amax = np.abs(b).max(-1, keepdims=True)
    scale = np.where(amax < TINY, 1.0, amax / E4M3_MAX)
    return np.where(amax < TINY, 0.0, b / scale).reshape(v.shape), scale[..., 0]


def e4m3_rne(v):
    return torch.from_numpy(v).to(torch.float8_e4m3fn).to(torch.float64).numpy()


def check_codes(q, scale, want, block, rel, what):
    """Codes and scales of `want` [T, n] in blocks of `block` columns.  The scales agree to
    `rel`; each code is a nearest e4m3 number of want / scale, where want's own relative
    error `rel` (and the scale's) may move it past the middle between two codes."""
    v, s = quantize(want, block)
    got_s = np64(scale).reshape(s.shape)
    close(got_s, s, rel * s, what + " scale")
    got = np64(q)
    best = e4m3_rne(v)
    off = np.abs(np.abs(got - v) - np.abs(best - v))
    assert np.array_equal(np.isnan(got), np.isnan(v)), what + ": NaN codes"
    slack = 4 * rel * np.abs(v)
    bad = ~(off <= slack) & ~np.isnan(v)
    assert not bad.any(), f"{what}: {bad.sum()} codes are not the nearest"


# ---------------------------------------------------------------------------------------
def norm(x, residual, weight, eps):
    h = x if residual is None else x + residual
    rstd = 1 / np.sqrt((h * h).mean(-1) + eps)
    return h, rstd, h * rstd[:, None] * weight


def norm_backward(dy, h, weight, rstd, dresidual):
    n = h.shape[1]
    xhat = h * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - xhat * (g * xhat).sum(-1, keepdims=True) / n)
    return dx if dresidual is None else dx + dresidual, (dy * xhat).sum(0)


def route(x, bias, k, sigmoid_score, groups, top_groups, group_top, renorm, scale):
    """ids and weights, one token at a time."""
    T, E = x.shape
    ids, weights = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        row = x[t]
        live = row != -np.inf
        if not live.any():
            continue
        if sigmoid_score:
            score = sigmoid(row)
        else:
            e = np.where(live, np.exp(row - row[live].max()), 0.0)
            score = e / e.sum()
        choice = np.where(live, score + (0 if bias is None else bias), -np.inf)
        if not sigmoid_score and bias is None and group_top == 1:
            choice = row
        if groups > 1:
            worth = []
            for g in range(groups):
                best = sorted(choice[g * (E // groups):(g + 1) * (E // groups)], reverse=True)
                best = [b for b in best[:group_top] if b != -np.inf]
                worth.append(sum(best) if best else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            group_of = np.arange(E) // (E // groups)
            choice = np.where(np.isin(group_of, kept), choice, -np.inf)
        order = [e for e in sorted(range(E), key=lambda e: (-choice[e], e)) if choice[e] > -np.inf]
        chosen = order[:k]
        w = score[chosen]
        if renorm and len(chosen):
            w = w / (w.sum() + (1e-20 if sigmoid_score else 0))
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = scale * w
    return ids, weights


def route_weights(x, ids, sigmoid_score, renorm, scale):
    """The weights of given ids as a function of the logits (for differences)."""
    here = (ids >= 0) & (ids < x.shape[1])
    at = np.where(here, ids, 0)
    if sigmoid_score:
        score = sigmoid(x)
    else:
        e = np.exp(x - x.max(-1, keepdims=True))
        score = e / e.sum(-1, keepdims=True)
    w = np.take_along_axis(score, at, 1) * here
    if renorm:
        w = w / np.maximum(w.sum(-1, keepdims=True), 1e-300)
    return scale * w


def route_backward(dw, x, ids, sigmoid_score, renorm, scale):
    T, E = x.shape
    d = np.zeros((T, E))
    for t in range(T):
        sel = [(j, i) for j, i in enumerate(ids[t]) if 0 <= i < E]
        if sigmoid_score:
            s = sigmoid(x[t])
            ds = np.zeros(E)
            total = sum(s[i] for _, i in sel) + 1e-20 if renorm else 1.0
            dot = sum(dw[t, j] * s[i] for j, i in sel) / total if renorm else 0.0
            for j, i in sel:
                ds[i] += scale * (dw[t, j] - dot) / total
            d[t] = ds * s * (1 - s)
        else:
            e = np.exp(x[t] - x[t].max())
            p = e / e.sum()
            if renorm:
                total = sum(p[i] for _, i in sel)
                dot = sum(dw[t, j] * p[i] / total for j, i in sel)
                for j, i in sel:
                    d[t, i] += scale * p[i] / total * (dw[t, j] - dot)
            else:
                dot = sum(dw[t, j] * p[i] for j, i in sel)
                d[t] = -scale * p * dot
                for j, i in sel:
                    d[t, i] += scale * p[i] * dw[t, j]
    return d


def dispatch(ids, E):
    """(m_sizes, dest, source token of each row) by a loop over the experts."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    dest, source, m = np.full(T * k, -1, np.int64), [], np.zeros(E, np.int64)
    for e in range(E):
        for i in np.nonzero(flat == e)[0]:
            dest[i] = len(source)
            source.append(i // k)
            m[e] += 1
    return m, dest.reshape(T, k), np.array(source, np.int64)


def combine(rows, dest, weights):
    T, k = dest.shape
    out, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= dest[t, j] < rows.shape[0]:
                w = 1.0 if weights is None else weights[t, j]
                out[t] += w * rows[dest[t, j]]
                size[t] += np.abs(w * rows[dest[t, j]])
    return out, size


def swiglu(x):
    gate, up = np.split(x, 2, axis=1)
    return gate * sigmoid(gate) * up


def swiglu_backward(dy, x):
    gate, up = np.split(x, 2, axis=1)
    s = sigmoid(gate)
    return np.concatenate([dy * up * s * (1 + gate * (1 - s)), dy * gate * s], axis=1)
