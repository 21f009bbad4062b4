"""The operators together: the example's mixture-of-experts block, forward and backward, against
the same block in 64 bits on the values of the e4m3 weights.

Each activation or gradient row that goes into a product is rounded to e4m3 (relative error of
an element uniform in +-2^-4 at most: 3.6 % in the root of the mean square, and independent
from element to element).  Forward two of them lie one behind the other, and the checkpoint
does not matter: 5.1 %, with the bf16 roundings 6 %.  Backward the SwiGLU's input comes from
the forward's rounded rows and its 8-bit checkpoint, and two more gradients are rounded: five
in all, 8 %, with bf16 and the two copies of the weights (each rounded to e4m3 by itself:
3.6 % twice more) 12 %."""
import os
import sys

import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
import moe_reference as ref
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import np64

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


def values(weight):
    return np64(weight[0]) * np64(weight[1])[..., None]


@pytest.mark.parametrize("T,H,W,E,k", [(1, 256, 128, 8, 2), (37, 512, 256, 16, 4),
                                       (300, 384, 128, 5, 3)])
def test_block(T, H, W, E, k):
    import moe_block as mb
    w = mb.make_weights(H, W, E, seed=T)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + 1)
    x, res, dout, dres = (torch.randn((T, H), generator=g, device="cuda").bfloat16()
                          for _ in range(4))
    out, stream, kept = mb.forward(w, x, res, k)
    grads = mb.backward(w, kept, dout, dres)
    torch.cuda.synchronize()
    assert fx.device_status() == 0

    norm, router, up, down = np64(w.norm), np64(w.router), values(w.up), values(w.down)
    h, rstd, y = ref.norm(np64(x), np64(res), norm, 1e-6)
    assert off(stream, h) < 2.0 ** -8
    ids = np64(kept.routing.ids)          # near-ties are the kernel's to decide
    assert ((ids >= 0) & (ids < E)).all()
    logits = y @ router.T
    weights = ref.route_weights(logits, ids, True, True, 1.0)
    m, dest, source = ref.dispatch(ids, E)
    assert np.array_equal(np64(kept.packed.m_sizes), m)
    assert np.array_equal(np64(kept.packed.dest), dest)
    expert = np.repeat(np.arange(E), m)
    gate_up = np.einsum("rh,rnh->rn", y[source], up[expert])
    rows = np.einsum("rw,rhw->rh", ref.swiglu(gate_up), down[expert])
    want, _ = ref.combine(rows, dest, weights)
    assert off(out, want) < 0.06

    # backward, from the 64-bit forward
    do = np64(dout)
    drows, dw = np.zeros_like(rows), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            drows[dest[t, j]] = weights[t, j] * do[t]
            dw[t, j] = do[t] @ rows[dest[t, j]]
    dgu = ref.swiglu_backward(np.einsum("rh,rhw->rw", drows, down[expert]), gate_up)
    dpacked = np.einsum("rn,rnh->rh", dgu, up[expert])
    dlogits = ref.route_backward(dw, logits, ids, True, True, 1.0)
    dy, _ = ref.combine(dpacked, dest, None)
    dy = dy + dlogits @ router
    dx, dnorm = ref.norm_backward(dy, h, norm, rstd, np64(dres))
    assert off(grads["x"], dx) < 0.12
    assert off(grads["norm"], dnorm) < 0.12
    assert off(grads["router"], dlogits.T @ y) < 0.12


def test_block_without_training_state():
    """Serving: no checkpoint and no rstd, the same output."""
    import moe_block as mb
    w = mb.make_weights(256, 128, 8)
    x = torch.randn((9, 256), device="cuda").bfloat16()
    a, _, kept = mb.forward(w, x, x, 2)
    b, _, served = mb.forward(w, x, x, 2, training=False)
    assert torch.equal(a, b)
    assert served.act.saved is None and served.norm.rstd is None
