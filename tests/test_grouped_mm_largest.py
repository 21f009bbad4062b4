"""The 16-bit products on the GPU with as many rows as a call may have (2^30)."""
import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import close, np64, rounding

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
MOST = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


@pytest.fixture(autouse=True)
def _status():
    torch.cuda.empty_cache()
    fx.device_status()
    yield
    torch.cuda.empty_cache()


def sizes(counts):
    return torch.tensor(counts, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("counts,owner", [([MOST, MOST], [0, 0, 0]), ([MOST - 5, 9, MOST], [0, 1, 1])])
def test_counts_past_the_largest_number_of_rows(counts, owner):
    """Clamped as in shorter calls: nothing behind the last row is written.  (owner: the experts of
    row 70001 and of the last two.)"""
    n = k = 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.zeros((MOST, k), dtype=BF16, device="cuda")
    rows = [70001, MOST - 2, MOST - 1]
    x[rows] = torch.randn((3, k), generator=g, device="cuda").to(BF16)
    w = torch.randn((len(counts), n, k), generator=g, device="cuda").to(BF16)
    whole = torch.full((MOST + 4096, n), 3.0, dtype=BF16, device="cuda")
    out = whole[:MOST]
    fx.grouped_mm(x, w, sizes(counts), out=out)
    assert fx.device_status() == fx.MSLKB_DEV_MSIZES_CLAMPED
    assert (whole[MOST:] == 3.0).all()
    for r, e in zip(rows, owner):
        a, b = np64(x[r]), np64(w[e])
        want = b @ a
        close(np64(out[r]), want, k * 2.0 ** -23 * (np.abs(b) @ np.abs(a)) + rounding(BF16, want),
              f"row {r}")
    out[rows] = 0
    assert not any(out[i:i + (1 << 26)].any() for i in range(0, MOST, 1 << 26))


@pytest.mark.parametrize("grad", [FP32, BF16])
def test_one_expert_with_all_rows(grad):
    """More tiles than CTA pairs, and one of them with 2^30 rows: in parts, of which none takes as long
    as a wait of the kernel may.  Sums of ones: exact."""
    x = torch.ones((MOST, 1), dtype=BF16, device="cuda")
    dy = torch.ones_like(x)
    counts = [0] * 1024
    counts[3], counts[700] = 40, MOST - 40
    dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts), dtype=grad)
    assert fx.device_status() == 0
    want = torch.tensor(counts, dtype=torch.float64).to(grad)
    assert torch.equal(dw.flatten().cpu(), want)


def test_long_rows():
    """A contraction of 2^25, turned and not, in parts; sums of ones."""
    k, n, g = 1 << 25, 8, 160
    x = torch.ones((g, k), dtype=BF16, device="cuda")
    w = torch.zeros((g, n, k), dtype=BF16, device="cuda")
    w[:, 3] = 1.0
    w[7, 5, -1] = 2.0
    ms = sizes([1] * g)
    want = torch.zeros((g, n))
    want[:, 3] = k
    want[7, 5] = 2.0
    out = fx.grouped_mm(x, w, ms)
    assert fx.device_status() == 0
    assert torch.equal(out.cpu(), want.to(BF16))
    w = w.view(g, k, n).zero_()
    w[:, :, 3] = 1.0
    w[7, -1, 5] = 2.0
    out = fx.grouped_mm(x, w, ms, transposed=True)
    assert fx.device_status() == 0
    assert torch.equal(out.cpu(), want.to(BF16))
