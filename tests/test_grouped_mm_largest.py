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
