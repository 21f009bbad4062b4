"""The norm of gradients and their clipping on the GPU: bounds and norms that are infinite or zero."""
import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


# a list of one cluster, one of several launches' size
SIZES = [[100, 3], [3_000_000, 70]]


def both_ways(grads, max_norm, **kw):
    """Clipped beside and in place: the same; -> (norm, results)."""
    r = fx.clip_grad_norm(grads, max_norm, **kw)
    held = [g.clone() for g in grads]
    norm = torch.zeros((), device="cuda")
    fx.clip_grad_norm(held, max_norm, out=(norm, held), **kw)
    for a, b in zip(held, r.grads):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(norm.view(torch.int32), r.norm.view(torch.int32))
    return r.norm.item(), r.grads


@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("sizes", SIZES)
def test_no_bound(sizes, inf):
    """An infinite bound leaves gradients as they are whatever their norm, unless that is NaN."""
    kind = INF if inf else 2.0
    for dtype in (BF16, FP16, FP32):
        grads = [torch.randn(n, device="cuda").to(dtype) for n in sizes]
        grads[0][5] = -INF
        for max_norm in (INF, 1e300):       # (past fp32's largest number: no bound either)
            norm, got = both_ways(grads, max_norm, norm_type=kind)
            assert norm == INF and all(torch.equal(a, b) for a, b in zip(got, grads))
        grads[0][5] = NAN
        norm, got = both_ways(grads, INF, norm_type=kind)
        assert np.isnan(norm) and all(torch.isnan(g).all() for g in got)


@pytest.mark.parametrize("sizes", SIZES)
def test_norm_past_fp32(sizes):
    """Finite gradients whose norm is not: left as they are without a bound, else scaled by 0."""
    grads = [torch.randn(n, device="cuda") for n in sizes]
    grads[0][:8] = 2.0 ** 127
    norm, got = both_ways(grads, INF)
    assert norm == INF and all(torch.equal(a, b) for a, b in zip(got, grads))
    norm, got = both_ways(grads, 1.0)
    assert norm == INF and not any(g.any() for g in got)


@pytest.mark.parametrize("sizes", SIZES)
def test_nothing_over_nothing(sizes):
    """Norm, bound and eps zero: nothing to clip."""
    grads = [torch.zeros(n, device="cuda") for n in sizes]
    norm, got = both_ways(grads, 0.0, eps=0.0)
    assert norm == 0 and not any(g.any() for g in got)
    grads[1][0] = 1.0
    norm, got = both_ways(grads, 0.0, eps=0.0)
    assert norm == 1 and not any(g.any() for g in got)
    # at the bound itself nothing changes
    norm, got = both_ways(grads, 1.0, eps=0.0)
    assert norm == 1 and all(torch.equal(a, b) for a, b in zip(got, grads))
