"""A mixture-of-experts block, forward and backward, on the library's operators.

    python examples/moe_block.py [--tokens 4096] [--hidden 7168] [--width 2048]
                                 [--experts 32] [--top-k 8]

norm + e4m3 rows -> router's logits -> experts and weights -> rows packed by expert
  -> grouped gate/up product -> SwiGLU + e4m3 rows (checkpoint of its input in 8 bits)
  -> grouped down product -> weighted sum per token

and back: the gradients of the tokens, the residual, the norm's weight and the router.  The
experts' weights stay as they are (e4m3, one scale per row, with a transposed copy for the
products of the backward pass); weights and inputs are random.
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


def backward(w, kept, dout, dresidual):
    """Gradients of out and of the residual stream -> dict of those of x (and of residual), the
    norm's weight and the router."""
    n, logits, r, d, a, rows = kept
    drows, dweights = fx.moe_combine_backward(dout, rows, d.dest, r.weights)
    da = product(*quantize_rows(drows), w.down_t, d.m_sizes)
    dgate_up = fx.swiglu_quant_backward(da, a.saved, a.saved_scale)
    dpacked = product(*quantize_rows(dgate_up), w.up_t, d.m_sizes)
    dlogits = fx.route_experts_backward(dweights, logits, r.ids, score="sigmoid").bfloat16()
    dy = fx.moe_combine(dpacked, d.dest) + dlogits @ w.router
    dx, dnorm = fx.add_rms_norm_quant_backward(dy, n.residual, w.norm, n.rstd, dresidual)
    return {"x": dx, "norm": dnorm, "router": dlogits.t() @ n.y}


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=8)
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
    flags = fx.device_status()
    if flags:
        raise SystemExit(f"device status {flags:#x}")


if __name__ == "__main__":
    main()
