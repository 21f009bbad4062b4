"""How well the sums of the 16-bit products keep what is added to them.

The tensor core's fp32 sums lose the bits below their last place, always towards zero, so it sums
1024 terms (64 steps of 16) at most, for fp32 gradients 512, and such sums are added with rounding.
The inputs here cancel: the terms of the second half of a period are those of the first, negated, so
that every result is exactly zero (or what is added), and 16 bits show what the sums lost.

Tolerance: 64 (32) steps that lose at most 2^-23 of what their terms add up to, and for each such
sum (and each part of a contraction) a rounding, at most 2^-24 of the largest sum, half a period's;
then the result's own.
"""
import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import close, np64, rounding

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


@pytest.fixture(autouse=True)
def _status():
    fx.device_status()
    yield
    assert fx.device_status() == 0


def positive(seed, *shape, dtype):
    """Values from 0.5 to 1."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda").mul_(0.5).add_(0.5).to(dtype)


def twice(t, dim, negate):
    return torch.cat([t, -t if negate else t], dim)


def sizes(counts):
    return torch.tensor(counts, dtype=torch.int64, device="cuda")


def lost(dtype, terms, magnitudes, period, parts=1):
    """Of sums of `terms` whose magnitudes add up to these, for results of a type."""
    each = 512 if dtype == FP32 else 1024
    roundings = (-(-terms // each) + parts) * 2.0 ** -24
    return (each / 16 * 2.0 ** -23 + roundings * period / (2 * terms)) * magnitudes


def parts_of(workspace_bytes, elements):
    assert workspace_bytes % (4 * elements) == 0
    return workspace_bytes // (4 * elements) or 1


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("n,k,period,split", [(10240, 32768, 32768, False), (10239, 8192, 8192, False),
                                              (72, 524288, 32768, True)])
def test_products(n, k, period, split, transposed, dtype):
    counts = [3, 0, 40, 1]
    m, g = sum(counts), len(counts)
    x = twice(positive(1, m, period // 2, dtype=dtype), 1, False).repeat(1, k // period)
    half = positive(2, g, *((period // 2, n) if transposed else (n, period // 2)), dtype=dtype)
    dim = 1 if transposed else 2
    w = twice(half, dim, True).repeat(*(k // period if d == dim else 1 for d in range(3)))
    if n % 8 == 0:
        p = parts_of(fx.mslkb_grouped_mm_workspace_bytes(256, 256, m, g, n, k, k, transposed), m * n)
        assert (p > 1) == split
    out = fx.grouped_mm(x, w, sizes(counts), transposed=transposed)
    at = 0
    for e, c in enumerate(counts):
        v = half[e].double() if transposed else half[e].double().t()
        mag = 2 * k / period * (x[at:at + c, :period // 2].double() @ v)
        tol = lost(dtype, k, np64(mag), period, 16) * (1 + 2.0 ** -8)
        close(np64(out[at:at + c]), np.zeros_like(tol), tol, f"expert {e}")
        at += c


def halves(seed, counts, width, negate, dtype):
    """Rows by expert, the second half of each expert's as the first (or negated)."""
    each = []
    for i, c in enumerate(counts):
        rows = twice(positive(seed + i, c // 2, width, dtype=dtype), 0, negate)
        each.append(rows)
    return torch.cat(each)


@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (FP16, FP16), (BF16, FP32)])
@pytest.mark.parametrize("add", [None, "aligned", "off 16 bytes"])
@pytest.mark.parametrize("counts,n,k", [([32768], 4096, 2560), ([32768] + [16] * 255, 256, 256),
                                        ([40, 8192, 0, 4] * 40, 250, 264)])
def test_weight_grad(counts, n, k, add, dtype, grad):
    """Experts that all have many rows, and one or a few with many beside others with few."""
    m, g = sum(counts), len(counts)
    assert fx.mslkb_grouped_mm_weight_grad_workspace_bytes(256, 256, m, g, 256, 256, 256, 256) == 0 \
        or g == 1
    dy, x = halves(1, counts, n, True, dtype), halves(1000, counts, k, False, dtype)
    before = None
    if add is not None:
        flat = torch.empty(g * n * k + 1, dtype=grad, device="cuda")
        before = flat[1:] if add == "off 16 bytes" else flat[:-1]
        before = before.view(g, n, k)
        before.copy_(positive(3, g, n, k, dtype=grad).mul_(2.0 ** -6))
    dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=before, dtype=grad)
    ends = np.cumsum(counts)
    for e in {0, 1, g // 2 + 1, g - 1} & set(range(g)):
        b = ends[e]
        a = b - counts[e]
        mag = np64(dy[a:b].abs().double().t() @ x[a:b].double())
        want = np.zeros((n, k)) if before is None else np64(before[e])
        tol = lost(grad, max(counts[e], 1), mag, counts[e])
        tol = tol + 2.0 ** -24 * (np.abs(want) + tol)
        close(np64(dw[e]), want, tol + rounding(grad, np.abs(want) + tol), f"expert {e}")
