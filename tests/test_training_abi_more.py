"""C entry points for training the experts, without a GPU: calls at the ends of what the sizes may
be."""
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from test_moe_abi import P, refused
from test_training_abi import GRADS, OUTS, clip, mm, weight_grad

MOST = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fxbuild.build()
    fx.lib()


@pytest.mark.parametrize("total,G,N,K", [
    (8, 1024, MOST, MOST), (8, 1, MOST, MOST), (MOST, 1, 2048, 8), (MOST, 1, 8, 2048),
    (8, 1024, 1 << 16, (1 << 14) + 1), (MOST, 1024, MOST, MOST)])
def test_sizes_whose_products_are_too_large(total, G, N, K):
    """Refused whatever the workspace, and before it is reckoned with: 64 bits would not hold the
    bytes of 1024 x 2^30 x 2^30 elements (nor of their rows of one less, copied)."""
    for workspace, nbytes in ((None, 0), (P, 1 << 62)):
        for less in (0, 1):
            kw = dict(total_M=total, G=G, N=N, K=K - less, workspace=workspace, bytes=nbytes)
            # (one less keeps three of the products above the limit)
            if total * N <= 1 << 40 and total * (K - less) <= 1 << 40 and \
                    G * N * (K - less) <= 1 << 40:
                continue
            refused(mm, fx.MSLKB_ERR_SHAPE, {**kw, "ldx": K, "transposed": 0},
                    {**kw, "ldx": K, "transposed": 1})
            refused(weight_grad, fx.MSLKB_ERR_SHAPE, {**kw, "ldx": K, "lddy": N})
            for t in (0, 1):
                assert fx.mslkb_grouped_mm_workspace_bytes(P, P, total, G, N, K - less, K, t) == 0
            assert fx.mslkb_grouped_mm_weight_grad_workspace_bytes(
                P, P, total, G, N, K - less, N, K) == 0


def test_workspace_of_the_largest_sizes():
    """Bytes of copies and slices at the limit: positive, and enough."""
    f = fx.mslkb_grouped_mm_workspace_bytes
    rows = 1 << 29
    assert f(P + 2, P + 2, rows, 1, 8, 2048, 2048, 0) >= 2 * rows * 2048
    assert f(P, P, rows, 1, 8, 2047, 2047, 0) >= 2 * rows * 2048
    assert f(P + 2, P, 1, 1024, 1 << 15, 1 << 15, 1 << 15, 1) >= 2 * 1 << 15
    f = fx.mslkb_grouped_mm_weight_grad_workspace_bytes
    assert f(P + 2, P + 2, MOST, 1, 512, 1024, 512, 1024) >= 2 * MOST * (512 + 1024)


def test_no_contraction_outlasts_a_wait():
    """Parts of at most 2^24 terms, whatever the number of tiles: a wait lasts as long as a part."""
    f = fx.mslkb_grouped_mm_weight_grad_workspace_bytes
    copies = 2 * MOST * 8 * 2                      # rows of one element, copied to 16 bytes
    assert f(P, P, MOST, 1024, 1, 1, 1, 1) == copies + 64 * 1024 * 4
    assert f(P, P, 1 << 25, 1024, 8, 8, 8, 8) == 2 * 1024 * 64 * 4
    assert f(P, P, (1 << 24) + 1, 1024, 8, 8, 8, 8) == 2 * 1024 * 64 * 4
    assert f(P, P, 1 << 24, 1024, 8, 8, 8, 8) == 0
    f = fx.mslkb_grouped_mm_workspace_bytes
    assert f(P, P, 200, 200, 8, 1 << 26, 1 << 26, 0) == 4 * 200 * 8 * 4
    assert f(P, P, 200, 200, 8, 1 << 24, 1 << 24, 0) == 0
    assert f(P, P, 1, 1, 8, MOST, MOST, 0) == 64 * 8 * 4


# addresses far from each other, which no call here follows
X, W, DY, OUT, COUNTS = ((i + 1) << 40 for i in range(5))


def test_products_over_their_inputs():
    """A result that shares a byte with an element of an input is refused."""
    kw = dict(total_M=8, G=2, N=64, K=64, ldx=64, x=X, w=W, m_sizes=COUNTS, out=OUT)
    out = 2 * 8 * 64

    def bad(fn, **more):
        refused(fn, fx.MSLKB_ERR_SHAPE, {**kw, **more})
    for t in (0, 1):
        for at, nbytes in ((X, 8 * 64 * 2), (W, 2 * 64 * 64 * 2), (COUNTS, 16)):
            for o in (at, at + nbytes - 2, at - out + 2):
                bad(mm, out=o, transposed=t)
    kw = dict(total_M=8, G=2, N=64, K=64, ldx=64, lddy=64, x=X, dy=DY, m_sizes=COUNTS, add=None)
    for wide in (0, 1):
        dw = 2 * 64 * 64 * (4 if wide else 2)
        for at, nbytes in ((X, 8 * 64 * 2), (DY, 8 * 64 * 2), (COUNTS, 16)):
            for o in (at, at + nbytes - 4, at - dw + 4):
                bad(weight_grad, dw=o, dw_fp32=wide)


@pytest.mark.skipif(torch.cuda.is_available(), reason="these calls reach the device where there is one")
def test_products_beside_their_inputs():
    """Right before and behind them, and between strided rows: taken, as far as the missing device."""
    other = mm(total_M=8, G=2, N=64, K=64, ldx=64, x=X, w=W, m_sizes=COUNTS, out=OUT)
    assert other in (fx.MSLKB_ERR_DEVICE, fx.MSLKB_ERR_CUDA)
    kw = dict(total_M=8, G=2, N=64, K=64, x=X, w=W, m_sizes=COUNTS)
    out = 2 * 8 * 64
    ld = 4096
    refused(mm, other, {**kw, "ldx": 64, "out": X - out}, {**kw, "ldx": 64, "out": X + 2 * 8 * 64},
            {**kw, "ldx": 64, "out": W - out}, {**kw, "ldx": 64, "out": W + 2 * 2 * 64 * 64},
            {**kw, "ldx": 64, "out": COUNTS - out}, {**kw, "ldx": 64, "out": COUNTS + 16},
            {**kw, "ldx": ld, "out": X + 128}, {**kw, "ldx": ld, "out": X + 2 * ld - out},
            {**kw, "ldx": ld, "out": X + 2 * 7 * ld + 128})
    refused(mm, fx.MSLKB_ERR_SHAPE, {**kw, "ldx": ld, "out": X + 126},
            {**kw, "ldx": ld, "out": X + 2 * ld - out + 2}, {**kw, "ldx": ld, "out": X + 2 * 7 * ld})


def test_norm_over_a_list():
    """The clipping's norm inside a gradient (10 bf16 at 256, 100 fp32 at 4096) or a result."""
    for at in (256, 272, 4096, 4492, 16384, 16400, 32768, 33164):
        refused(clip, fx.MSLKB_ERR_SHAPE, {"norm": at})
        refused(clip, fx.MSLKB_ERR_SHAPE, {"norm": at, "outs": GRADS if at < 8192 else OUTS})
