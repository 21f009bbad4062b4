"""A mixture-of-experts block, forward and backward, on the library's operators.

    python examples/moe_block.py [--tokens 4096] [--hidden 7168] [--width 2048]
                                 [--experts 32] [--top-k 8] [--train STEPS]

norm + e4m3 rows -> router's logits -> experts and weights -> rows packed by expert
  -> grouped gate/up product -> SwiGLU + e4m3 rows (checkpoint of its input in 8 bits)
  -> grouped down product -> weighted sum per token

and back: the gradients of the tokens, the residual, the norm's weight and the router.  The
experts' weights stay as they are (e4m3, one scale per row, with a transposed copy for the
products of the backward pass); weights and inputs are random.

With --train the experts are trained as well: they are kept in bf16 besides, which the products of
the backward pass take as they are, their gradients come from products over each expert's rows, all
gradients are clipped together, and the e4m3 weights are made again after every step.
"""
from __future__ import annotations

import argparse
import os
import sys
from typing import NamedTuple

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fp8_rowwise_scaled_gb300 as fx  # noqa: E402
from fp8_rowwise_scaled_gb300.synthetic import quantize_rows  # noqa: E402


class Weights(NamedTuple):
    norm: torch.Tensor            # [H]
    router: torch.Tensor          # [E, H] bf16
    bias: torch.Tensor            # [E] fp32, for balance
    up: tuple                     # [E, 2W, H] e4m3 and scales [E, 2W]
    down: tuple                   # [E, H, W]
    up_t: tuple                   # [E, H, 2W]
    down_t: tuple                 # [E, W, H]


class Experts(NamedTuple):
    """The experts' weights in 16 bits, for training them."""
    up: torch.Tensor              # [E, 2W, H]
    down: torch.Tensor            # [E, H, W]


class Kept(NamedTuple):
    """What the backward pass needs of the forward pass."""
    norm: fx.NormQuant
    logits: torch.Tensor
    routing: fx.Routing
    packed: fx.Dispatch
    act: fx.SwigluQuant
    rows: torch.Tensor


def make_weights(hidden, width, experts, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def randn(*shape, scale=1.0):
        return scale * torch.randn(shape, generator=g, device=device)

    def pair(n, k):   # an expert's matrix and its transposed copy, each quantised per row
        m = [randn(n, k, scale=k ** -0.5) for _ in range(experts)]
        straight = [quantize_rows(v) for v in m]
        turned = [quantize_rows(v.t().contiguous()) for v in m]
        return [tuple(torch.stack(x) for x in zip(*q)) for q in (straight, turned)]

    up, up_t = pair(2 * width, hidden)
    down, down_t = pair(hidden, width)
    return Weights((1 + 0.1 * randn(hidden)).bfloat16(),
                   randn(experts, hidden, scale=hidden ** -0.5).bfloat16(),
                   0.05 * randn(experts), up, down, up_t, down_t)


def make_experts(hidden, width, experts, seed=0, device="cuda", dtype=torch.bfloat16):
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def stack(n, k):
        return torch.stack([k ** -0.5 * torch.randn((n, k), generator=g, device=device)
                            for _ in range(experts)]).to(dtype)
    return Experts(stack(2 * width, hidden), stack(hidden, width))


def quantised(w, experts):
    """w with the e4m3 copies of these experts' weights."""
    def pair(m):
        def rows(v):
            q, scale = quantize_rows(v.reshape(-1, v.shape[-1]))
            return q.reshape(v.shape), scale.reshape(v.shape[:2])
        return rows(m), rows(m.transpose(1, 2).contiguous())
    (up, up_t), (down, down_t) = pair(experts.up), pair(experts.down)
    return w._replace(up=up, down=down, up_t=up_t, down_t=down_t)


def product(xq, x_scale, weight, m_sizes):
    q, scale = weight
    return fx.f8f8bf16_rowwise_grouped_stacked(xq, q, x_scale, scale, m_sizes)


def forward(w, x, residual, top_k, training=True):
    """x, residual [T, H] bf16 -> (out [T, H], the residual stream [T, H], Kept)."""
    experts = w.router.shape[0]
    n = fx.add_rms_norm_quant(x, w.norm, residual, want_y=True, want_rstd=training)
    logits = (n.y @ w.router.t()).float()
    r = fx.route_experts(logits, top_k, bias=w.bias, score="sigmoid")
    d = fx.moe_dispatch(n.q, n.scale, r.ids, experts)
    gate_up = product(d.x, d.x_scale, w.up, d.m_sizes)
    a = fx.swiglu_quant(gate_up, checkpoint=training)
    rows = product(a.q, a.scale, w.down, d.m_sizes)
    out = fx.moe_combine(rows, d.dest, r.weights)
    return out, n.residual, Kept(n, logits, r, d, a, rows)


def backward(w, kept, dout, dresidual, experts=None):
    """Gradients of out and of the residual stream -> dict of those of x (and of residual), the
    norm's weight and the router; with the experts' 16-bit weights those of up and down as well
    (fp32), and products in 16 bits throughout."""
    n, logits, r, d, a, rows = kept
    drows, dweights = fx.moe_combine_backward(dout, rows, d.dest, r.weights)
    more = {}
    if experts is None:
        da = product(*quantize_rows(drows), w.down_t, d.m_sizes)
    else:
        act = (a.q.float() * a.scale.unsqueeze(-1)).to(drows.dtype)
        more["down"] = fx.grouped_mm_weight_grad(drows, act, d.m_sizes)
        da = fx.grouped_mm(drows, experts.down, d.m_sizes, transposed=True)
    dgate_up = fx.swiglu_quant_backward(da, a.saved, a.saved_scale)
    if experts is None:
        dpacked = product(*quantize_rows(dgate_up), w.up_t, d.m_sizes)
    else:
        packed = fx.moe_dispatch(n.y, None, r.ids, experts.up.shape[0]).x
        more["up"] = fx.grouped_mm_weight_grad(dgate_up, packed, d.m_sizes)
        dpacked = fx.grouped_mm(dgate_up, experts.up, d.m_sizes, transposed=True)
    dlogits = fx.route_experts_backward(dweights, logits, r.ids, score="sigmoid").bfloat16()
    dy = fx.moe_combine(dpacked, d.dest) + dlogits @ w.router
    dx, dnorm = fx.add_rms_norm_quant_backward(dy, n.residual, w.norm, n.rstd, dresidual)
    return {"x": dx, "norm": dnorm, "router": dlogits.t() @ n.y, **more}


def train_step(w, experts, x, residual, dout, dresidual, top_k, lr, max_norm=1.0):
    """One step of gradient descent on the weights, the gradients of all of them clipped together
    -> (Weights, Experts, the gradients' norm)."""
    _, _, kept = forward(w, x, residual, top_k)
    grads = backward(w, kept, dout, dresidual, experts)
    names = ("norm", "router", "up", "down")
    each = [grads[k] for k in names]
    norm, clipped = fx.clip_grad_norm(each, max_norm,
                                      out=(torch.empty((), device=x.device), each))
    old = (w.norm, w.router, experts.up, experts.down)
    new = [(v.float() - lr * g.float()).to(v.dtype) for v, g in zip(old, clipped)]
    experts = Experts(*new[2:])
    return quantised(w._replace(norm=new[0], router=new[1]), experts), experts, norm


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--train", type=int, default=0, metavar="STEPS")
    a = ap.parse_args()
    w = make_weights(a.hidden, a.width, a.experts)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, res, dout, dres = (torch.randn((a.tokens, a.hidden), generator=g, device="cuda").bfloat16()
                          for _ in range(4))
    for _ in range(3):   # warm up
        out, stream, kept = forward(w, x, res, a.top_k)
        backward(w, kept, dout, dres)
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    marks[0].record()
    out, stream, kept = forward(w, x, res, a.top_k)
    marks[1].record()
    grads = backward(w, kept, dout, dres)
    marks[2].record()
    torch.cuda.synchronize()
    counts = kept.packed.m_sizes
    print(f"{a.tokens} tokens x {a.hidden}, {a.experts} experts of {a.width}, top {a.top_k}: "
          f"{int(counts.min())}-{int(counts.max())} rows per expert; forward "
          f"{marks[0].elapsed_time(marks[1]):.2f} ms, backward "
          f"{marks[1].elapsed_time(marks[2]):.2f} ms")
    print(f"|out| {out.float().norm():.1f}  " +
          "  ".join(f"|d {k}| {v.float().norm():.4g}" for k, v in grads.items()))
    if a.train:
        experts = make_experts(a.hidden, a.width, a.experts)
        w = quantised(w, experts)
        for step in range(a.train):
            w, experts, norm = train_step(w, experts, x, res, dout, dres, a.top_k, 1e-2)
            print(f"step {step}: gradients' norm {norm.item():.4g}")
    flags = fx.device_status()
    if flags:
        raise SystemExit(f"device status {flags:#x}")


if __name__ == "__main__":
    main()
