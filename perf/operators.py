"""Cases for measuring the operators around the FP8 grouped GEMM in a mixture-of-experts block.

Each operator has a plain form here (elementary torch operations in 32 bits, rounded once at the
end), a call of the library's own kernel, and an evaluation in 64 bits from its definition:

* norm: residual addition, root-mean-square norm and an e4m3 output with its scales (the
  activations of the gate/up product), and the gradient;
* route: each token's experts and weights from the router's logits, and the gradient;
* dispatch / combine: the routed rows packed by expert with their counts (the stacked layout),
  the weighted sum of the experts' rows per token, and its gradient;
* swiglu: silu(gate) * up with an e4m3 output (the activations of the down product), with an
  e4m3 checkpoint of the input in training, and the gradient from that checkpoint.

``own`` selects the library's kernels; a case is a dict of plain values.
"""
import torch

own = False

EPS = 1e-6
BLOCK = 128           # elements per scale in the block-scaled (groupwise) layouts
E4M3_MAX = 448.0
TINY = 2.0 ** -80     # rows (or blocks) whose largest magnitude is below this are stored as zeros

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    """4 to 12 cases over the real range: hidden size 7168 with experts of width 2048 (the
    gate/up and down products of the DS-V3-shaped workloads), 8 experts per token."""
    return [
        # one token of a decode step; the router reads y beside the quantised row
        {"name": "norm_decode_1", "op": "norm", "tokens": 1, "hidden": 7168, "dtype": "bf16",
         "residual": True, "groupwise": False, "y": True, "rstd": False},
        # a prefill or training micro-batch, scales per block, everything the backward needs
        {"name": "norm_prefill_8192", "op": "norm", "tokens": 8192, "hidden": 7168,
         "dtype": "bf16", "residual": True, "groupwise": True, "y": True, "rstd": True},
        # the same micro-batch backwards, with the gradient that arrives on the residual
        {"name": "norm_backward_8192", "op": "norm_backward", "tokens": 8192, "hidden": 7168,
         "dtype": "bf16", "residual": True},
        # a small decode batch: sigmoid scores with a balance bias, 4 of 8 groups
        {"name": "route_decode_16", "op": "route", "tokens": 16, "experts": 256, "top_k": 8,
         "dtype": "fp32", "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4,
         "group_top": 2, "renormalize": True},
        # the same router over a long prefill
        {"name": "route_prefill_16384", "op": "route", "tokens": 16384, "experts": 256,
         "top_k": 8, "dtype": "fp32", "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "group_top": 2, "renormalize": True},
        # training with softmax scores that are not renormalised: every logit has a gradient
        {"name": "route_backward_16384", "op": "route_backward", "tokens": 16384,
         "experts": 160, "top_k": 6, "dtype": "bf16", "score": "softmax", "groups": 1,
         "top_groups": 1, "group_top": 1, "bias": False, "renormalize": False},
        # a decode batch on a device that holds 32 of the experts: most choices live elsewhere
        {"name": "dispatch_decode_32", "op": "dispatch", "tokens": 32, "top_k": 8,
         "experts": 32, "hidden": 7168, "groupwise": False, "elsewhere": 0.75},
        # a prefill with every expert here, scales per block
        {"name": "dispatch_prefill_8192", "op": "dispatch", "tokens": 8192, "top_k": 8,
         "experts": 256, "hidden": 7168, "groupwise": True, "elsewhere": 0.0},
        # the experts' rows of an uneven micro-batch summed back per token
        {"name": "combine_8111", "op": "combine", "tokens": 8111, "top_k": 8, "experts": 256,
         "hidden": 7168, "dtype": "bf16", "elsewhere": 0.0},
        # its gradient: the experts' rows' and the routing weights'
        {"name": "combine_backward_4096", "op": "combine_backward", "tokens": 4096, "top_k": 8,
         "experts": 64, "hidden": 7168, "dtype": "bf16", "elsewhere": 0.0},
        # training forward: the input of the activation is kept in 8 bits
        {"name": "swiglu_checkpoint_32768", "op": "swiglu", "rows": 32768, "width": 2048,
         "dtype": "bf16", "groupwise": True, "checkpoint": True},
        # and read back for its gradient
        {"name": "swiglu_backward_32768", "op": "swiglu_backward", "rows": 32768,
         "width": 2048, "dtype": "bf16", "checkpoint": True},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case: sizes over their whole range (tokens from one up, odd and ragged sizes
    among them), every type, form and direction."""
    op = rng.choice(["norm", "norm", "norm_backward", "route", "route", "route_backward",
                     "dispatch", "dispatch", "combine", "combine_backward", "swiglu",
                     "swiglu_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("route", "route_backward"):
        experts = rng.choice([8, 16, 31, 64, 128, 160, 256, 384, 500])
        score = rng.choice(["sigmoid", "softmax"])
        groups = rng.choice([g for g in (1, 2, 4, 8) if experts % g == 0 and experts // g >= 2])
        top_groups = rng.randint(1, groups)
        reach = experts // groups * top_groups
        tokens = _log_uniform(rng, 1, 16384)
        # (one choice of one token, renormalised, is always 1)
        top_k = rng.randint(1 if tokens >= 64 else 2, min(reach, rng.choice([2, 8, 8, 10])))
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "dtype": dtype,
                "score": score, "bias": score == "sigmoid" and rng.random() < 0.7,
                "groups": groups, "top_groups": top_groups,
                "group_top": 1 if score == "softmax" else rng.choice([1, 2]),
                "renormalize": rng.random() < 0.6}
    if op in ("dispatch", "combine", "combine_backward"):
        top_k = rng.choice([1, 2, 4, 6, 8])
        hidden = rng.choice([256, 1000, 2048, 4096, 5120, 7168, 8192])
        groupwise = op == "dispatch" and hidden % BLOCK == 0 and rng.random() < 0.5
        size = 1 if op == "dispatch" else 4 if dtype == "fp32" else 2
        most = 900_000_000 // ((2 * top_k + 1) * hidden * size)
        tokens = _log_uniform(rng, 1, min(16384, most))
        # (a handful of tokens may have no expert here at all: nothing to measure)
        case = {"op": op, "tokens": tokens, "top_k": top_k,
                "experts": rng.choice([8, 16, 32, 60, 128, 256]), "hidden": hidden,
                "elsewhere": rng.choice([0.0, 0.0, 0.5, 0.9]) if tokens >= 64 else 0.0}
        case.update({"groupwise": groupwise} if op == "dispatch" else {"dtype": dtype})
        return case
    if op in ("norm", "norm_backward"):
        hidden = rng.choice([128, 1000, 1025, 2048, 4096, 5120, 7168, 8192, 16384])
        most = 150_000_000 // (hidden * (2 if dtype == "fp32" else 1))
        case = {"op": op, "tokens": _log_uniform(rng, 1, min(16384, most)), "hidden": hidden,
                "dtype": dtype, "residual": rng.random() < 0.7}
        if op == "norm":
            case.update({"groupwise": hidden % BLOCK == 0 and rng.random() < 0.5,
                         "y": rng.random() < 0.5, "rstd": rng.random() < 0.5})
        return case
    width = rng.choice([128, 1000, 768, 2048, 4096, 8192])
    whole = width % BLOCK == 0
    most = 100_000_000 // (width * (2 if dtype == "fp32" else 1))
    case = {"op": op, "rows": _log_uniform(rng, 1, min(65536, most)), "width": width,
            "dtype": dtype, "checkpoint": whole and rng.random() < 0.6}
    if op == "swiglu":
        case["groupwise"] = whole and rng.random() < 0.5
    return case


def work(case):
    """Bytes that one pass has to read and write (each input and output once) and its
    floating-point operations."""
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case.get("dtype", "bf16")]
    if op in ("route", "route_backward"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        if op == "route":
            return {"bytes": t * e * size + 8 * t * k + (4 * e if case["bias"] else 0),
                    "flops": 4 * t * e}
        return {"bytes": 2 * t * e * size + 8 * t * k, "flops": 6 * t * e}
    if op == "norm":
        t, h = case["tokens"], case["hidden"]
        streams = 1 + 2 * case["residual"] + case["y"]
        scales = h // BLOCK if case["groupwise"] else 1
        return {"bytes": t * h * (streams * size + 1) + h * size
                + 4 * t * (scales + case["rstd"]), "flops": 7 * t * h}
    if op == "norm_backward":
        t, h = case["tokens"], case["hidden"]
        return {"bytes": t * h * (3 + case["residual"]) * size + 4 * t + h * (size + 4),
                "flops": 10 * t * h}
    if op in ("swiglu", "swiglu_backward"):
        r, w = case["rows"], case["width"]
        kept = r * (2 * w + 4 * (2 * w // BLOCK))
        if op == "swiglu":
            scales = w // BLOCK if case["groupwise"] else 1
            return {"bytes": r * w * (2 * size + 1) + 4 * r * scales
                    + (kept if case["checkpoint"] else 0), "flops": 8 * r * w}
        return {"bytes": r * w * 3 * size + (kept if case["checkpoint"] else 2 * r * w * size),
                "flops": 12 * r * w}
    t, k, h = case["tokens"], case["top_k"], case["hidden"]
    here = t * k * (1.0 - case["elsewhere"])      # rows of this device's experts, on average
    if op == "dispatch":
        row = h + 4 * (h // BLOCK if case["groupwise"] else 1)
        read = t * (1.0 - case["elsewhere"] ** k) * row
        return {"bytes": read + here * row + 8 * t * k + 8 * case["experts"], "flops": 0}
    if op == "combine":
        return {"bytes": here * h * size + t * h * size + 8 * t * k, "flops": 2 * here * h}
    return {"bytes": 2 * here * h * size + t * h * size + 12 * t * k, "flops": 3 * here * h}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _choices(case, gen):
    """[tokens, top_k] int32 experts: distinct per token, popularity Zipf(1.1) as in the MoE
    workloads; a choice that lives on another device is -1."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    rank = torch.arange(1, e + 1, device="cuda", dtype=torch.float32)
    gumbel = -torch.log(-torch.log(torch.rand((t, e), generator=gen, device="cuda")
                                   .clamp(1e-7, 1 - 1e-7)))
    ids = torch.topk(gumbel - 1.1 * torch.log(rank), k, dim=1).indices.to(torch.int32)
    away = torch.rand((t, k), generator=gen, device="cuda") < case["elsewhere"]
    return torch.where(away, torch.full_like(ids, -1), ids)


def _packed(ids, experts):
    """Row of every choice when the choices are packed by expert, in token order; -1 where
    the choice is not here."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    order = torch.sort(key, stable=True).indices
    dest = torch.empty_like(flat)
    dest[order] = torch.arange(flat.numel(), device=flat.device)
    return torch.where(flat < 0, torch.full_like(flat, -1), dest).to(torch.int32) \
        .reshape(ids.shape)


def _empty(*shape, dtype):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    """Inputs and output buffers on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case.get("dtype", "bf16")]
    f32, e4m3 = torch.float32, torch.float8_e4m3fn
    s = {"case": dict(case), "op": op}
    if op in ("norm", "norm_backward"):
        t, h = case["tokens"], case["hidden"]
        # hidden states: rows of different sizes, norm weights around one
        size = torch.exp(0.5 * _randn(gen, t, 1))
        s["weight"] = (1.0 + 0.2 * _randn(gen, h)).to(dt)
        if op == "norm":
            s["x"] = _randn(gen, t, h).mul_(size).to(dt)
            s["residual"] = _randn(gen, t, h).mul_(3 * size).to(dt) if case["residual"] else None
            scales = (t, h // BLOCK) if case["groupwise"] else (t,)
            s["out"] = (_empty(t, h, dtype=e4m3), _empty(*scales, dtype=f32),
                        _empty(t, h, dtype=dt) if case["residual"] else None,
                        _empty(t, h, dtype=dt) if case["y"] else None,
                        _empty(t, dtype=f32) if case["rstd"] else None)
        else:
            s["h"] = _randn(gen, t, h).mul_(3 * size).to(dt)
            s["rstd"] = s["h"].float().square().mean(-1).add(EPS).rsqrt()
            s["dy"] = _randn(gen, t, h).to(dt)
            s["dresidual"] = _randn(gen, t, h).to(dt) if case["residual"] else None
            s["out"] = (_empty(t, h, dtype=dt), _empty(h, dtype=f32))
    elif op in ("route", "route_backward"):
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        # logits of a trained router: experts differ in popularity
        s["logits"] = (1.5 * _randn(gen, t, e) + 0.5 * _randn(gen, e)).to(dt)
        s["bias"] = 0.1 * _randn(gen, e) if case["bias"] else None
        if op == "route":
            s["out"] = (_empty(t, k, dtype=torch.int32), _empty(t, k, dtype=f32))
        else:
            s["ids"] = _route(s["logits"], s["bias"], case)[0]
            s["dweights"] = _randn(gen, t, k)
            s["out"] = _empty(t, e, dtype=dt)
    elif op in ("dispatch", "combine", "combine_backward"):
        t, k, h = case["tokens"], case["top_k"], case["hidden"]
        s["ids"] = _choices(case, gen)
        if op == "dispatch":
            blocks = h // BLOCK if case["groupwise"] else 1
            x = _randn(gen, t, blocks, h // blocks)
            s["x_scale"] = (x.abs().amax(-1) / E4M3_MAX).reshape((t, blocks) if
                                                                 case["groupwise"] else (t,))
            s["xq"] = (x / (x.abs().amax(-1, keepdim=True) / E4M3_MAX)).reshape(t, h).to(e4m3)
            s["out"] = (_empty(t * k, h, dtype=e4m3),
                        _empty(*((t * k, blocks) if case["groupwise"] else (t * k,)), dtype=f32),
                        _empty(case["experts"], dtype=torch.int64),
                        _empty(t, k, dtype=torch.int32))
        else:
            s["dest"] = _packed(s["ids"], case["experts"])
            s["rows"] = _randn(gen, t * k, h).to(dt)
            s["weights"] = torch.softmax(_randn(gen, t, k), -1)
            if op == "combine":
                s["out"] = _empty(t, h, dtype=dt)
            else:
                s["dout"] = _randn(gen, t, h).to(dt)
                s["out"] = (_empty(t * k, h, dtype=dt), _empty(t, k, dtype=f32))
    else:
        r, w = case["rows"], case["width"]
        # the gate/up product's rows
        x = _randn(gen, r, 2 * w).mul_(torch.exp(0.5 * _randn(gen, r, 1)))
        if op == "swiglu":
            s["x"] = x.to(dt)
            scales = (r, w // BLOCK) if case["groupwise"] else (r,)
            kept = case["checkpoint"]
            s["out"] = (_empty(r, w, dtype=e4m3), _empty(*scales, dtype=f32),
                        _empty(r, 2 * w, dtype=e4m3) if kept else None,
                        _empty(r, 2 * w // BLOCK, dtype=f32) if kept else None)
        else:
            s["dy"] = _randn(gen, r, w).to(dt)
            if case["checkpoint"]:
                b = x.reshape(r, 2 * w // BLOCK, BLOCK)
                s["saved_scale"] = b.abs().amax(-1) / E4M3_MAX
                s["saved"] = (b / s["saved_scale"].unsqueeze(-1)).to(e4m3).reshape(r, 2 * w)
            else:
                s["saved"], s["saved_scale"] = x.to(dt), None
            s["out"] = _empty(r, 2 * w, dtype=dt)
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _quantize(v, block):
    """e4m3 codes and fp32 scales (largest magnitude / 448) of each block of `block` columns."""
    t, h = v.shape
    b = v.reshape(t, h // block, block)
    amax = b.abs().amax(-1, keepdim=True)
    zero = amax < TINY
    scale = torch.where(zero, torch.ones_like(amax), amax / E4M3_MAX)
    q = torch.where(zero, torch.zeros_like(b), b / scale)
    return q.reshape(t, h).to(torch.float8_e4m3fn), scale.reshape(t, h // block)


def _norm(s, case):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    y = h * rstd * s["weight"].float()
    q, scale = _quantize(y, BLOCK if case["groupwise"] else case["hidden"])
    dt = s["x"].dtype
    return {"q": q, "scale": scale if case["groupwise"] else scale.reshape(-1),
            "residual": h.to(dt) if case["residual"] else None,
            "y": y.to(dt) if case["y"] else None,
            "rstd": rstd.reshape(-1) if case["rstd"] else None}


def _norm_backward(s, case):
    xhat = s["h"].float() * s["rstd"].unsqueeze(-1)
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = s["rstd"].unsqueeze(-1) * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xhat).sum(0)}


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _first(v, n):
    """Indices of the n largest values of each row, the lowest index first among equals."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :n]


def _route(logits, bias, case):
    lowest = float("-inf")
    x = logits.float()
    t, e = x.shape
    softmax = case["score"] == "softmax"
    top = x.amax(-1, keepdim=True)
    if softmax and bias is None and case["group_top"] == 1:
        choice = x                      # the softmax keeps the logits' order
    else:
        score = torch.exp(x - top) if softmax else _sigmoid(x)
        if softmax:
            score = score / score.sum(-1, keepdim=True)
        choice = score if bias is None else score + bias
        choice = torch.where(x == lowest, torch.full_like(choice, lowest), choice)
    groups, per = case["groups"], e // case["groups"]
    if groups > 1:
        best = torch.sort(choice.reshape(t, groups, per), dim=-1, descending=True).values
        best = best[..., :case["group_top"]]
        rest = torch.where(best[..., 1:] == lowest, torch.zeros_like(best[..., 1:]),
                           best[..., 1:])
        worth = best[..., 0] + rest.sum(-1)
        kept = torch.zeros_like(worth, dtype=torch.bool)
        kept.scatter_(1, _first(worth, case["top_groups"]), True)
        choice = torch.where(kept.repeat_interleave(per, dim=1), choice,
                             torch.full_like(choice, lowest))
    ids = _first(choice, case["top_k"])
    there = choice.gather(1, ids) != lowest
    sel = x.gather(1, ids)
    if softmax:
        if case["renormalize"]:
            w = torch.where(there, torch.exp(sel - sel.amax(-1, keepdim=True)),
                            torch.zeros_like(sel))
            w = w / w.sum(-1, keepdim=True)
        else:
            w = torch.exp(sel - top) / torch.exp(x - top).sum(-1, keepdim=True)
    else:
        w = torch.where(there, _sigmoid(sel), torch.zeros_like(sel))
        if case["renormalize"]:
            w = w / (w.sum(-1, keepdim=True) + 1e-20)
    w = torch.where(there, w, torch.zeros_like(w))
    return torch.where(there, ids, torch.full_like(ids, -1)).to(torch.int32), w


def _route_backward(s, case):
    x, ids, g = s["logits"].float(), s["ids"].long(), s["dweights"]
    here = ids >= 0
    at = torch.where(here, ids, torch.zeros_like(ids))
    g = torch.where(here, g, torch.zeros_like(g))
    sel = torch.where(here, x.gather(1, at), torch.full_like(g, float("-inf")))
    if case["score"] == "softmax":
        if case["renormalize"]:
            p = torch.exp(sel - sel.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            d = p * (g - (p * g).sum(-1, keepdim=True))
            dx = torch.zeros_like(x)
        else:
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            chosen = torch.where(here, p.gather(1, at), torch.zeros_like(g))
            dx = -p * (chosen * g).sum(-1, keepdim=True)
            d = chosen * g
    else:
        sig = torch.where(here, _sigmoid(sel), torch.zeros_like(g))
        if case["renormalize"]:
            total = sig.sum(-1, keepdim=True) + 1e-20
            d = (g - (g * sig).sum(-1, keepdim=True) / total) / total
        else:
            d = g
        d = d * sig * (1.0 - sig)
        dx = torch.zeros_like(x)
    d = torch.where(here, d, torch.zeros_like(d))
    return dx.scatter_add_(1, at, d).to(s["logits"].dtype)


def _dispatch(s, case):
    ids, e = s["ids"], case["experts"]
    t, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, e), flat)
    order = torch.sort(key, stable=True).indices
    dest = torch.empty_like(flat)
    dest[order] = torch.arange(t * k, device=flat.device)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=flat.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    here = torch.arange(t * k, device=flat.device) < counts[:e].sum()
    rows = torch.where(here.unsqueeze(-1), s["xq"].view(torch.uint8)[order // k],
                       torch.zeros((), dtype=torch.uint8, device=flat.device))
    scale = s["x_scale"][order // k]
    scale = torch.where(here.reshape(-1, *[1] * (scale.dim() - 1)), scale,
                        torch.zeros_like(scale))
    return {"xq": rows.view(torch.float8_e4m3fn), "x_scale": scale, "m_sizes": counts[:e],
            "dest": torch.where(flat < 0, torch.full_like(flat, -1), dest).to(torch.int32)
            .reshape(t, k)}


def _combine(s, case):
    dest = s["dest"].long()
    here = (dest >= 0).unsqueeze(-1)
    rows = s["rows"][dest.clamp(min=0).reshape(-1)].float().reshape(*dest.shape, -1)
    rows = torch.where(here, rows, torch.zeros((), device=rows.device))
    return (rows * s["weights"].unsqueeze(-1)).sum(1).to(s["rows"].dtype)


def _combine_backward(s, case):
    dest = s["dest"].long()
    here = dest >= 0
    t, k = dest.shape
    dout = s["dout"].float()
    rows = s["rows"][dest.clamp(min=0).reshape(-1)].float().reshape(t, k, -1)
    dweights = (rows * dout.unsqueeze(1)).sum(-1)
    dweights = torch.where(here, dweights, torch.zeros_like(dweights))
    each = (dout.unsqueeze(1) * s["weights"].unsqueeze(-1)).to(s["rows"].dtype)
    drows = torch.zeros((t * k + 1, dout.shape[1]), dtype=s["rows"].dtype, device=dout.device)
    at = torch.where(here, dest, torch.full_like(dest, t * k)).reshape(-1)
    drows[at] = each.reshape(t * k, -1)
    return {"drows": drows[:t * k], "dweights": dweights}


def _swiglu(s, case):
    w = case["width"]
    x = s["x"].float()
    gate, up = x[:, :w], x[:, w:]
    q, scale = _quantize(gate / (1.0 + torch.exp(-gate)) * up,
                         BLOCK if case["groupwise"] else w)
    kept = _quantize(x, BLOCK) if case["checkpoint"] else (None, None)
    return {"q": q, "scale": scale if case["groupwise"] else scale.reshape(-1),
            "saved": kept[0], "saved_scale": kept[1]}


def _swiglu_backward(s, case):
    w = case["width"]
    x = s["saved"].float()
    if s["saved_scale"] is not None:
        x = (x.reshape(-1, 2 * w // BLOCK, BLOCK) * s["saved_scale"].unsqueeze(-1)) \
            .reshape(-1, 2 * w)
    gate, up, dy = x[:, :w], x[:, w:], s["dy"].float()
    sig = _sigmoid(gate)
    dgate = dy * up * sig * (1.0 + gate * (1.0 - sig))
    return torch.cat([dgate, dy * gate * sig], dim=1).to(s["dy"].dtype)


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "norm":
        return _norm(s, case)
    if op == "norm_backward":
        return _norm_backward(s, case)
    if op == "route":
        ids, w = _route(s["logits"], s["bias"], case)
        return {"ids": ids, "weights": w}
    if op == "route_backward":
        return _route_backward(s, case)
    if op == "dispatch":
        return _dispatch(s, case)
    if op == "combine":
        return _combine(s, case)
    if op == "combine_backward":
        return _combine_backward(s, case)
    return _swiglu(s, case) if op == "swiglu" else _swiglu_backward(s, case)


# ---------------------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------------------
def _own(s):
    import fp8_rowwise_scaled_gb300 as fx
    case, op, out = s["case"], s["op"], s["out"]
    if op == "norm":
        q, scale, residual, y, rstd = fx.add_rms_norm_quant(
            s["x"], s["weight"], s["residual"], eps=EPS, groupwise=case["groupwise"],
            want_y=case["y"], want_rstd=case["rstd"], out=out)
        return {"q": q, "scale": scale, "residual": residual if case["residual"] else None,
                "y": y, "rstd": rstd}
    if op == "norm_backward":
        dx, dweight = fx.add_rms_norm_quant_backward(s["dy"], s["h"], s["weight"], s["rstd"],
                                                     s["dresidual"], out=out)
        return {"dx": dx, "dweight": dweight}
    if op == "route":
        ids, w = fx.route_experts(
            s["logits"], case["top_k"], bias=s["bias"], score=case["score"],
            num_groups=case["groups"], topk_groups=case["top_groups"],
            group_top=case["group_top"], renormalize=case["renormalize"], out=out)
        return {"ids": ids, "weights": w}
    if op == "route_backward":
        return fx.route_experts_backward(s["dweights"], s["logits"], s["ids"],
                                         score=case["score"],
                                         renormalize=case["renormalize"], out=out)
    if op == "dispatch":
        xq, x_scale, m_sizes, dest = fx.moe_dispatch(s["xq"], s["x_scale"], s["ids"],
                                                     case["experts"], out=out)
        return {"xq": xq, "x_scale": x_scale, "m_sizes": m_sizes, "dest": dest}
    if op == "combine":
        return fx.moe_combine(s["rows"], s["dest"], s["weights"], out=out)
    if op == "combine_backward":
        drows, dweights = fx.moe_combine_backward(s["dout"], s["rows"], s["dest"],
                                                  s["weights"], out=out)
        return {"drows": drows, "dweights": dweights}
    if op == "swiglu":
        q, scale, saved, saved_scale = fx.swiglu_quant(
            s["x"], groupwise=case["groupwise"], checkpoint=case["checkpoint"], out=out)
        return {"q": q, "scale": scale, "saved": saved, "saved_scale": saved_scale}
    return fx.swiglu_quant_backward(s["dy"], s["saved"], s["saved_scale"], out=out)


def run(state):
    """One pass through the operator, and its outputs."""
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _codes64(v, block):
    """v / scale before the rounding to e4m3, and the scales, in 64 bits."""
    rows = v.reshape(v.shape[0], -1, block)
    largest = rows.abs().max(dim=2).values
    scale = largest / 448
    scale[largest < TINY] = 1
    rows = rows / scale[:, :, None]
    rows[largest < TINY] = 0
    return rows.reshape(v.shape), scale


def _per_row(case, scale):
    return scale if case["groupwise"] else scale[:, 0]


def _exact_norm(s, case):
    v = s["x"].double()
    if case["residual"]:
        v = v.add_(s["residual"].double())
    r = (torch.linalg.vecdot(v, v) / v.shape[1] + EPS) ** -0.5
    y = s["weight"].double()[None, :] * r[:, None] * v
    codes, scale = _codes64(y, BLOCK if case["groupwise"] else case["hidden"])
    return {"q": codes, "scale": _per_row(case, scale),
            "residual": v if case["residual"] else None, "y": y if case["y"] else None,
            "rstd": r if case["rstd"] else None}


def _exact_norm_backward(s, case):
    v, w, dy, r = (s[n].double() for n in ("h", "weight", "dy", "rstd"))
    # y_i = w_i r v_i and dr/dv_j = -r^3 v_j / n
    along = torch.linalg.vecdot(dy * w, v) * r ** 3 / v.shape[1]
    dx = dy * w * r[:, None] - along[:, None] * v
    if case["residual"]:
        dx += s["dresidual"].double()
    return {"dx": dx, "dweight": torch.einsum("ti,ti,t->i", dy, v, r)}


def _exact_route(s, case):
    """The weights in 64 bits for the choice of the 32-bit scores (a choice between scores that
    agree to 32 bits is the plain form's)."""
    ids = _route(s["logits"], s["bias"], case)[0].long()
    x = s["logits"].double()
    score = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
    w = torch.take_along_dim(score, ids.clamp(min=0), 1) * (ids >= 0)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": None, "weights": w}


def _exact_route_backward(s, case):
    x = s["logits"].double().requires_grad_(True)
    score = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
    here = s["ids"] >= 0
    w = torch.take_along_dim(score, s["ids"].long().clamp(min=0), 1) * here
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    (w * s["dweights"].double()).sum().backward()
    return x.grad


def _exact_dispatch(s, case):
    ids = s["ids"].cpu().reshape(-1)
    k, rows = s["ids"].shape[1], []
    for e in range(case["experts"]):
        rows.append(torch.nonzero(ids == e)[:, 0])
    source = torch.cat(rows).to("cuda") // k
    xq = torch.zeros((ids.numel(), case["hidden"]), dtype=torch.float64, device="cuda")
    xq[:len(source)] = s["xq"].double()[source]
    scale = torch.zeros((ids.numel(), *s["x_scale"].shape[1:]), dtype=torch.float64,
                        device="cuda")
    scale[:len(source)] = s["x_scale"].double()[source]
    return {"xq": xq, "x_scale": scale, "m_sizes": None, "dest": None}


def _exact_combine(s, case):
    total = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device="cuda")
    for j in range(s["dest"].shape[1]):
        t = torch.nonzero(s["dest"][:, j] >= 0)[:, 0]
        total[t] += s["weights"][t, j, None].double() * s["rows"][s["dest"][t, j].long()].double()
    return total


def _exact_combine_backward(s, case):
    dest, dout = s["dest"], s["dout"].double()
    drows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
    dweights = torch.zeros(dest.shape, dtype=torch.float64, device="cuda")
    for j in range(dest.shape[1]):
        t = torch.nonzero(dest[:, j] >= 0)[:, 0]
        r = dest[t, j].long()
        drows[r] = s["weights"][t, j, None].double() * dout[t]
        dweights[t, j] = torch.linalg.vecdot(dout[t], s["rows"][r].double())
    return {"drows": drows, "dweights": dweights}


def _exact_swiglu(s, case):
    gate, up = s["x"].double().chunk(2, dim=1)
    q, scale = _codes64(torch.sigmoid(gate) * gate * up,
                        BLOCK if case["groupwise"] else case["width"])
    kept = _codes64(s["x"].double(), BLOCK) if case["checkpoint"] else (None, None)
    return {"q": q, "scale": _per_row(case, scale), "saved": kept[0], "saved_scale": kept[1]}


def _exact_swiglu_backward(s, case):
    x = s["saved"].double()
    if case["checkpoint"]:
        x = x * s["saved_scale"].double().repeat_interleave(BLOCK, dim=1)
    x.requires_grad_(True)
    gate, up = x.chunk(2, dim=1)
    torch.sum(gate * torch.sigmoid(gate) * up * s["dy"].double()).backward()
    return x.grad


def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits. Values that run()
    rounds (to e4m3, bf16 or fp16) are given before that rounding."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "route": _exact_route,
            "route_backward": _exact_route_backward, "dispatch": _exact_dispatch,
            "combine": _exact_combine, "combine_backward": _exact_combine_backward,
            "swiglu": _exact_swiglu, "swiglu_backward": _exact_swiglu_backward}[case["op"]](s, case)
