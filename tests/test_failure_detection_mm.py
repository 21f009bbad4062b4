"""Failure detection in the 16-bit products, without a GPU fault (as in test_failure_detection.py):
the first pair of CTAs of a launch withholds a stage of its pipeline, the wait for it runs out after
50 ms, the kernel records that in the device status word and returns; the call after it is right."""
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from test_grouped_mm import check_grad, check_mm, randn, sizes

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


def stalled_then_right(call, check):
    check(call())
    torch.cuda.synchronize()
    assert fx.device_status() == 0
    fx.mslkb_set_wait_timeout_us(50_000)
    try:
        fx.mslkb_test_stall_next_launch()
        call()
        again = call()      # right behind it
        torch.cuda.synchronize()
        assert fx.device_status() & fx.MSLKB_DEV_TIMEOUT
    finally:
        fx.mslkb_set_wait_timeout_us(0)
    check(again)
    check(call())
    torch.cuda.synchronize()
    assert fx.device_status() == 0


# short contractions, long ones, few tiles in parts, odd rows that are copied first and stored
# element by element
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,n,k", [([300, 0, 700, 33], 2048, 512), ([300, 0, 700, 33] * 8, 1024, 2048),
                                        ([40, 3], 512, 4096), ([300, 41] * 20, 1001, 1101)])
def test_products(counts, n, k, transposed):
    x = randn(1, sum(counts), k)
    w = randn(2, len(counts), *((k, n) if transposed else (n, k)))
    ms = sizes(counts)
    stalled_then_right(lambda: fx.grouped_mm(x, w, ms, transposed=transposed),
                       lambda out: check_mm(out, x, w, counts, transposed))


# experts with few rows, with many, with many beside few; ends of rows inside a step
@pytest.mark.parametrize("grad", [FP32, BF16])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("counts", [[64, 0, 75, 33] * 20, [1500, 901] * 40, [3000] + [5] * 99])
def test_weight_grad(counts, add, grad):
    n, k = 256, 512
    m = sum(counts)
    dy, x = randn(1, m, n), randn(2, m, k)
    before = randn(3, len(counts), n, k, dtype=grad) if add else None
    ms = sizes(counts)
    stalled_then_right(lambda: fx.grouped_mm_weight_grad(dy, x, ms, add=before, dtype=grad),
                       lambda dw: check_grad(dw, dy, x, counts, before))
