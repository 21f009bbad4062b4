"""How far each element of the routing gradient may be from its 64-bit value: the roundings of
the formula in fp32, u = 2^-24 each, relative to what the element is made of (an absolute bound
would be far above the values that a softmax over all experts leaves to those not chosen)."""
import numpy as np

from moe_reference import U, rounding, sigmoid


def route_backward_tolerance(dw, x, ids, sigmoid_score, renorm, scale, dtype, want):
    """dw [T, k], x [T, E] and ids [T, k] (distinct, outside [0, E): none) in 64 bits."""
    T, E = x.shape
    per_lane = next(p for p in (1, 2, 4, 5, 8, 12, 16, 32) if 32 * p >= E)
    here = (ids >= 0) & (ids < E)
    at = np.where(here, ids, 0)
    g = np.where(here, dw * scale, 0.0)
    sel = np.take_along_axis(x, at, 1)
    tol = np.zeros((T, E))

    def spread(v):          # [T, k] to the experts that were chosen
        out = np.zeros((T, E))
        for t, j in zip(*np.nonzero(here)):
            out[t, ids[t, j]] = v[t, j]
        return out

    if sigmoid_score:
        # sigmoid: the exponential 2, 1 + e, the division; a product each
        s, rest = np.where(here, sigmoid(sel), 0.0), sigmoid(-sel)
        if not renorm:
            tol = spread(12 * U * np.abs(g) * s * rest)
        else:
            total = s.sum(1, keepdims=True) + 1e-20                     # 4 + 5 additions
            along = np.abs(g * s).sum(1, keepdims=True) / total
            inner = np.abs(g - (g * s).sum(1, keepdims=True) / total)
            tol = spread(U * s * rest / total * (2 * np.abs(g) + 22 * along + 21 * inner))
    elif renorm:
        live = np.where(here, sel, -np.inf)
        top = live.max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        w = np.exp(live - top)
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
        off = np.where(w > 0, (np.abs(np.where(w > 0, live - top, 0.0)) + 2), 0.0) * U  # exp
        of_sum = (w * off).sum(1, keepdims=True) + 5 * U
        rel = off.max(1, keepdims=True) + of_sum + 2 * U
        dot = np.abs(w * g).sum(1, keepdims=True)
        tol = spread(w * (U * (2 * np.abs(g) + dot) + dot * (rel + 8 * U)) +
                     np.take_along_axis(np.abs(want), at, 1) * (rel + 2 * U))
    else:
        top = x.max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        p = np.exp(x - top)
        p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
        off = np.where(p > 0, np.abs(np.where(p > 0, x - top, 0.0)) + 2, 0.0) * U
        of_sum = (p * off).sum(1, keepdims=True) + (per_lane + 5) * U
        mine = np.where(here, np.take_along_axis(p, at, 1), 0.0) * np.abs(g)
        dot = mine.sum(1, keepdims=True)
        tol = p * dot * (off + off.max(1, keepdims=True) + 2 * of_sum + 12 * U)
        own = np.where(here, np.take_along_axis(off, at, 1), 0.0)
        tol = tol + spread(mine * (own + of_sum + 4 * U)) + U * np.abs(want)
    return tol + rounding(dtype, want)
