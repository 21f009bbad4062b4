"""C entry points for training the experts, without a GPU: argument errors come before any CUDA
call, empty calls do nothing."""
import ctypes

import pytest

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from fp8_rowwise_scaled_gb300 import moe
from test_moe_abi import P, call, refused


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fxbuild.build()
    fx.lib()


mm = call(fx.mslkb_grouped_mm, dict(
    x=P, w=P, m_sizes=P, out=P, total_M=8, G=2, N=64, K=64, ldx=64, transposed=0,
    dtype=moe.MSLKB_BF16, workspace=None, bytes=0, stream=0))
weight_grad = call(fx.mslkb_grouped_mm_weight_grad, dict(
    dy=P, x=P, m_sizes=P, add=P, dw=P, total_M=8, G=2, N=64, K=64, lddy=64, ldx=64,
    dtype=moe.MSLKB_BF16, dw_fp32=1, workspace=None, bytes=0, stream=0))
BIG = (1 << 30) + 1


def test_products_refuse():
    refused(mm, fx.MSLKB_ERR_NULL, *({k: None} for k in ("x", "w", "m_sizes", "out")))
    refused(mm, fx.MSLKB_ERR_SHAPE, {"total_M": -1}, {"G": -1}, {"N": -1}, {"K": -1}, {"ldx": 63},
            {"G": 1025}, {"total_M": BIG}, {"N": BIG}, {"K": BIG, "ldx": BIG}, {"ldx": 1 << 31})
    refused(mm, fx.MSLKB_ERR_DTYPE, {"dtype": moe.MSLKB_FP32}, {"dtype": 3}, {"dtype": -1})
    refused(mm, fx.MSLKB_ERR_ALIGN, {"x": 257}, {"w": 257}, {"out": 257}, {"m_sizes": 260})
    refused(weight_grad, fx.MSLKB_ERR_NULL, *({k: None} for k in ("dy", "x", "m_sizes", "dw")))
    refused(weight_grad, fx.MSLKB_ERR_SHAPE, {"total_M": -1}, {"G": -1}, {"N": -1}, {"K": -1},
            {"ldx": 63}, {"lddy": 63}, {"G": 1025}, {"total_M": BIG}, {"N": BIG, "lddy": BIG},
            {"K": BIG, "ldx": BIG}, {"ldx": 1 << 31}, {"lddy": 1 << 31},
            {"add": P + 4}, {"dw": P + 4 * 2 * 64 * 64 - 4})        # over a part of each other
    refused(weight_grad, fx.MSLKB_ERR_DTYPE, {"dtype": moe.MSLKB_FP32}, {"dtype": 7})
    refused(weight_grad, fx.MSLKB_ERR_ALIGN, {"x": 257}, {"dy": 257}, {"dw": 258}, {"add": 258},
            {"m_sizes": 260}, {"dw_fp32": 0, "dw": 257})


def test_products_workspace():
    """Copies of the operands whose rows are not aligned to 16 bytes."""
    f = fx.mslkb_grouped_mm_workspace_bytes
    assert f(P, P, 8, 2, 64, 64, 64, 0) == 0 and f(P, P, 8, 2, 64, 63, 64, 1) == 0
    assert f(P, P, 8, 2, 64, 63, 64, 0) == 2 * 64 * 64 * 2          # w's rows of 63
    assert f(P, P, 8, 2, 64, 64, 65, 0) == 8 * 64 * 2               # x's, 65 apart
    assert f(P + 2, P + 2, 8, 2, 64, 64, 64, 0) == 2 * 64 * 64 * 2 + 8 * 64 * 2
    assert f(P, P, 1, 1, 1, 64, 65, 0) == 0                         # one row of each
    assert f(P, P, 0, 2, 64, 63, 63, 0) == f(P, P, 8, 2, 64, -1, 63, 0) == 0
    refused(mm, fx.MSLKB_ERR_WORKSPACE, {"ldx": 65}, {"x": P + 2},
            {"ldx": 65, "workspace": P, "bytes": 1023}, {"ldx": 65, "workspace": P + 8,
                                                         "bytes": 1 << 20})
    f = fx.mslkb_grouped_mm_weight_grad_workspace_bytes
    assert f(P, P, 8, 2, 64, 64, 64, 64) == 0 and f(P, P, 8, 2, 64, 64, 65, 64) == 1024
    assert f(P, P, 8, 2, 64, 64, 64, 65) == 1024 and f(P, P, 0, 2, 64, 64, 65, 65) == 0
    # one expert's 64 x 64 sums of many rows: in slices
    assert f(P, P, 1 << 16, 1, 64, 64, 64, 64) % (64 * 64 * 4) == 0
    assert f(P, P, 1 << 16, 1, 64, 64, 64, 64) > 64 * 64 * 4
    refused(weight_grad, fx.MSLKB_ERR_WORKSPACE, {"ldx": 65}, {"dy": P + 2},
            {"lddy": 65, "workspace": P, "bytes": 1023})


def test_products_of_nothing():
    refused(mm, fx.MSLKB_OK, {"total_M": 0, "x": None, "out": None}, {"G": 0, "m_sizes": None},
            {"N": 0, "w": None})
    refused(weight_grad, fx.MSLKB_OK, {"G": 0, "dw": None}, {"N": 0}, {"K": 0, "dw": None})


def array(kind, *values):
    return (kind * len(values))(*values)


GRADS = array(ctypes.c_void_p, 256, 4096)
OUTS = array(ctypes.c_void_p, 16384, 32768)
SIZES = array(ctypes.c_int64, 10, 100)
TYPES = array(ctypes.c_int32, moe.MSLKB_BF16, moe.MSLKB_FP32)
norm = call(fx.mslkb_grad_norm, dict(
    grads=GRADS, sizes=SIZES, dtypes=TYPES, count=2, kind=0, norm=P, workspace=P, bytes=1 << 20,
    stream=0))
clip = call(fx.mslkb_clip_grad_norm, dict(
    grads=GRADS, outs=OUTS, sizes=SIZES, dtypes=TYPES, count=2, kind=0, max_norm=1.0, eps=1e-6,
    norm=P, workspace=P, bytes=1 << 20, stream=0))


def test_lists_refuse():
    bad_size, bad_type = array(ctypes.c_int64, 10, -1), array(ctypes.c_int32, 0, 3)
    for fn in (norm, clip):
        refused(fn, fx.MSLKB_ERR_NULL, *({k: None} for k in ("grads", "sizes", "dtypes", "norm")),
                {"grads": array(ctypes.c_void_p, 256, None)})
        refused(fn, fx.MSLKB_ERR_SHAPE, {"count": -1}, {"count": 65537}, {"kind": 2}, {"kind": -1},
                {"sizes": bad_size}, {"sizes": array(ctypes.c_int64, 1 << 41, 1)})
        refused(fn, fx.MSLKB_ERR_DTYPE, {"dtypes": bad_type})
        refused(fn, fx.MSLKB_ERR_ALIGN, {"grads": array(ctypes.c_void_p, 257, 4096)},
                {"grads": array(ctypes.c_void_p, 256, 4098)}, {"norm": 258})
        refused(fn, fx.MSLKB_ERR_WORKSPACE, {"workspace": None}, {"workspace": 264},
                {"bytes": 4095})
    refused(clip, fx.MSLKB_ERR_NULL, {"outs": None}, {"outs": array(ctypes.c_void_p, 16384, None)})
    refused(clip, fx.MSLKB_ERR_ALIGN, {"outs": array(ctypes.c_void_p, 16385, 32768)})
    refused(clip, fx.MSLKB_ERR_SHAPE, {"max_norm": -1.0}, {"max_norm": float("nan")},
            {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")},
            # one result over the other, a result over the other's gradient, or beside its own
            {"outs": array(ctypes.c_void_p, 16384, 16400)},
            {"outs": array(ctypes.c_void_p, 4096 + 396, 32768)},
            {"outs": array(ctypes.c_void_p, 258, 32768)})


def test_list_workspace():
    f = fx.mslkb_grad_norm_workspace_bytes
    assert f(0) == f(1) == f(1024) == 4096 and f(1025) == 8192 and f(-1) == f(65537) == 0
