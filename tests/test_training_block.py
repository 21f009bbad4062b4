"""The operators for training together: the example's mixture-of-experts block with its experts in
16 bits besides, its gradients against 64 bits and their clipping.

The rounding of rows to e4m3 is what the forward pass's own test counts: 6 % of out.  The
gradients of the experts' weights are sums over rows of products of what those rows give: of a
gradient in 16 bits that goes back through a SwiGLU whose input comes from the 8-bit checkpoint
of rounded rows (three roundings to e4m3 of 3.6 % each, 6.3 %), and of activations that were rounded
to e4m3 twice one behind the other (5.1 %): 8.1 %, with bf16 10 %.
"""
import os
import sys

import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
import moe_reference as ref
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import U, close, np64, rounding

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


def off(got, want):
    got = np64(got)
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def block(T, H, W, E, seed):
    import moe_block as mb
    experts = mb.make_experts(H, W, E, seed=seed)
    w = mb.quantised(mb.make_weights(H, W, E, seed=seed), experts)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    return mb, w, experts, [torch.randn((T, H), generator=g, device="cuda").bfloat16()
                            for _ in range(4)]


@pytest.mark.parametrize("T,H,W,E,k", [(1, 256, 128, 8, 2), (37, 512, 256, 16, 4),
                                       (300, 384, 128, 5, 3)])
def test_gradients(T, H, W, E, k):
    mb, w, experts, (x, res, dout, dres) = block(T, H, W, E, T)
    _, _, kept = mb.forward(w, x, res, k)
    grads = mb.backward(w, kept, dout, dres, experts)
    torch.cuda.synchronize()
    assert fx.device_status() == 0

    up, down = np64(experts.up), np64(experts.down)
    _, _, y = ref.norm(np64(x), np64(res), np64(w.norm), 1e-6)
    ids = np64(kept.routing.ids)
    weights = ref.route_weights(y @ np64(w.router).T, ids, True, True, 1.0)
    m, dest, source = ref.dispatch(ids, E)
    expert = np.repeat(np.arange(E), m)
    gate_up = np.einsum("rh,rnh->rn", y[source], up[expert])
    act = ref.swiglu(gate_up)
    drows = np.zeros((len(source), H))
    for t in range(T):
        for j in range(k):
            drows[dest[t, j]] = weights[t, j] * np64(dout)[t]
    dgu = ref.swiglu_backward(np.einsum("rh,rhw->rw", drows, down[expert]), gate_up)
    want_up, want_down = np.zeros_like(up), np.zeros_like(down)
    for r, e in enumerate(expert):
        want_up[e] += np.outer(dgu[r], y[source[r]])
        want_down[e] += np.outer(drows[r], act[r])
    assert grads["up"].dtype == grads["down"].dtype == torch.float32
    assert off(grads["up"], want_up) < 0.10
    assert off(grads["down"], want_down) < 0.10
    empty = torch.from_numpy(m == 0).cuda()
    assert not grads["up"][empty].any() and not grads["down"][empty].any()
    # the tokens' gradient: as the block's own in e4m3, with fewer roundings
    fewer = mb.backward(w, kept, dout, dres)
    assert off(grads["x"], np64(fewer["x"])) < 0.12


def test_step():
    """The step's norm is that of the gradients, its weights are the old ones less the clipped
    gradients."""
    mb, w, experts, (x, res, dout, dres) = block(64, 256, 128, 8, 5)
    _, _, kept = mb.forward(w, x, res, 2)
    grads = mb.backward(w, kept, dout, dres, experts)
    names = ("norm", "router", "up", "down")
    total = np.sqrt(sum((np64(grads[k]) ** 2).sum() for k in names))
    scale = 0.5 / (total + 1e-6)
    w2, e2, norm = mb.train_step(w, experts, x, res, dout, dres, 2, lr=1.0, max_norm=0.5)
    assert abs(norm.item() - total) <= 18 * U * total
    for got, old, name in ((w2.norm, w.norm, "norm"), (w2.router, w.router, "router"),
                           (e2.up, experts.up, "up"), (e2.down, experts.down, "down")):
        step = np64(grads[name]) * scale
        want = np64(old) - step
        # the clipped gradient, rounded to its type, taken from the old weight in fp32 and rounded
        tol = 21 * U * np.abs(step) + rounding(grads[name].dtype, step) + U * np.abs(want)
        close(np64(got), want, tol + rounding(got.dtype, np.abs(want) + tol), name)
    again = mb.train_step(w2, e2, x, res, dout, dres, 2, lr=1.0, max_norm=0.5)
    torch.cuda.synchronize()
    assert all(torch.isfinite(v).all() for v in (*again[1], again[2]))
    assert fx.device_status() == 0


def test_forward_in_16_bits_is_the_products():
    """grouped_mm on the packed rows against the block's own products (e4m3 rows and weights)."""
    mb, w, experts, (x, res, _, _) = block(50, 256, 128, 8, 9)
    n = fx.add_rms_norm_quant(x, w.norm, res, want_y=True)
    r = fx.route_experts((n.y @ w.router.t()).float(), 2)
    d = fx.moe_dispatch(n.q, n.scale, r.ids, 8)
    rows = fx.moe_dispatch(n.y, None, r.ids, 8).x
    full = fx.grouped_mm(rows, experts.up, d.m_sizes)
    # one rounding to e4m3 of either operand: 5.1 %
    assert off(mb.product(d.x, d.x_scale, w.up, d.m_sizes), np64(full)) < 0.06


def test_backward_in_a_graph():
    """A captured backward pass with clipping, replayed with other gradients of out, gives what the
    calls give."""
    mb, w, experts, (x, res, dout, dres) = block(48, 256, 128, 8, 3)
    _, _, kept = mb.forward(w, x, res, 2)

    def step():
        grads = mb.backward(w, kept, dout, dres, experts)
        each = [grads[k] for k in ("norm", "router", "up", "down")]
        return fx.clip_grad_norm(each, 0.1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    g = torch.Generator(device="cuda")
    for seed in range(3):
        g.manual_seed(seed)
        dout.copy_(torch.randn(dout.shape, generator=g, device="cuda"))
        graph.replay()
        want = step()
        assert torch.equal(held.norm, want.norm)
        assert all(torch.equal(a, b) for a, b in zip(held.grads, want.grads))
    assert fx.device_status() == 0


def test_host_threads():
    """Four host threads, each with products and a clipping of its own on a stream of its own."""
    import threading
    cases, errors = [], []
    for i in range(4):
        g = torch.Generator(device="cuda")
        g.manual_seed(i)
        m, n, k = 150 + 40 * i, 200 + i, 136 + 8 * i     # rows of odd and of aligned lengths
        cases.append([torch.randn(s, generator=g, device="cuda").bfloat16()
                      for s in ((m, k), (3, n, k), (m, n))] +
                     [torch.tensor([m - 100, 0, 90], device="cuda"),
                      torch.cuda.Stream(priority=-1)])

    def calls(x, w, dy, sizes, stream):
        out = fx.grouped_mm(x, w, sizes, stream=stream)
        dx = fx.grouped_mm(dy, w, sizes, transposed=True, stream=stream)
        dw = fx.grouped_mm_weight_grad(dy, x, sizes, stream=stream)
        return out, dx, dw, *fx.clip_grad_norm([dw, out, dx], 1.0, stream=stream).grads

    def worker(case, got):
        try:
            torch.cuda.set_device(0)
            for _ in range(20):
                got.append(calls(*case))
            case[-1].synchronize()
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))
    want = [calls(*c) for c in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    threads = [threading.Thread(target=worker, args=a) for a in zip(cases, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not any(t.is_alive() for t in threads) and not errors, errors
    for one, runs in zip(want, got):
        assert len(runs) == 20
        assert all(torch.equal(a, b) for r in runs for a, b in zip(r, one))
    assert fx.device_status() == 0
