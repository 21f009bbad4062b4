"""More of the operators around the grouped product on the GPU: what tests/test_moe_ops.py does
not reach, with its helpers and the same 64-bit forms."""
import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
import moe_reference as ref
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import U, close, np64, rounding
from test_moe_ops import BF16, EPS, FP16, FP32, gen, randn, shifted, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


@pytest.mark.parametrize("T,H", [(2900, 136), (3000, 264), (2000, 520), (1900, 1000), (1700, 1032),
                                 (1500, 2056), (900, 4104), (700, 5128), (800, 8192)])
@pytest.mark.parametrize("with_res", [True, False])
def test_norm_backward_fp32_many_rows_per_cta(T, H, with_res):
    """32-bit rows through the ring, several per CTA, most with a last warp partly past the row's
    end: right, and the same bits every time."""
    g = gen(T + H)
    dy, h, w = randn(g, T, H), randn(g, T, H, scale=2.0), randn(g, H)
    dres = randn(g, T, H) if with_res else None
    rstd = h.double().square().mean(-1).add(EPS).rsqrt().float()
    dx, dw = fx.add_rms_norm_quant_backward(dy, h, w, rstd, dres)
    a = [np64(t) for t in (dy, h, w, rstd)]
    want_dx, want_dw = ref.norm_backward(*a, None if dres is None else np64(dres))
    xhat, gg = a[1] * a[3][:, None], a[0] * a[2]
    size = a[3][:, None] * (np.abs(gg) + np.abs(xhat) * np.abs(gg * xhat).mean(-1, keepdims=True))
    close(dx, want_dx, 48 * U * size + 2 * U * np.abs(want_dx), "dx")
    # additions: a thread's rows, up to 16 rows side by side, up to 19 partial sums a warp, 32
    # warps; and the roundings of h * rstd and of the product
    close(dw, want_dw, (T // 152 + 1 + 16 + 19 + 32 + 2) * U * np.abs(a[0] * xhat).sum(0), "dweight")
    for _ in range(20):
        again = fx.add_rms_norm_quant_backward(dy, h, w, rstd, dres)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw), "not the same bits again"
