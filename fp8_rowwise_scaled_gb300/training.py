"""Operators for training the experts: their products in 16 bits, forward and backward.

    grouped_mm(x, w) -> ... -> grouped_mm(dy, w, transposed=True)     the input's gradient
                               grouped_mm_weight_grad(dy, x)          the weights' gradient

As in moe.py, whose conventions hold here too: ``mslkb_*`` functions mirror the C entry points,
the others take torch CUDA tensors, run on the current stream or on ``stream``, and put their
results into ``out`` where it is given.
"""
from __future__ import annotations

import ctypes

import fp8_rowwise_scaled_gb300 as _fx

from . import moe as _moe


def declare(L: ctypes.CDLL) -> ctypes.CDLL:
    """Argument and result types of this module's entry points on a loaded library."""
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    for name, args in {
            "mslkb_grouped_mm": [p] * 4 + [i64] * 5 + [i32, i32, p],
            "mslkb_grouped_mm_weight_grad": [p] * 5 + [i64] * 6 + [i32, i32, p]}.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    return L


# ---------------------------------------------------------------------------------------
# raw C entry points (integer pointers, None for NULL)
# ---------------------------------------------------------------------------------------
def mslkb_grouped_mm(x, w, m_sizes, out, total_M, G, N, K, ldx, transposed, dtype,
                     stream=0) -> int:
    return _fx.lib().mslkb_grouped_mm(x, w, m_sizes, out, total_M, G, N, K, ldx, transposed,
                                      dtype, stream)


def mslkb_grouped_mm_weight_grad(dy, x, m_sizes, add, dw, total_M, G, N, K, lddy, ldx, dtype,
                                 dw_fp32=1, stream=0) -> int:
    return _fx.lib().mslkb_grouped_mm_weight_grad(dy, x, m_sizes, add, dw, total_M, G, N, K, lddy,
                                                  ldx, dtype, dw_fp32, stream)


# ---------------------------------------------------------------------------------------
# torch front end
# ---------------------------------------------------------------------------------------
def _binding():
    if _moe._b is None:
        _moe._setup()
    return _moe._b


def _stack_shape(t, name):
    if not isinstance(t, _moe._torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name}: expected 3 dims, got {t.dim()}")
    return t.shape


def grouped_mm(x, w, m_sizes, *, transposed=False, out=None, stream=None):
    """out[r] = x[r] . w[g]^T for every row r of expert g, or x[r] . w[g] with ``transposed``.

    x [total_M, K] bf16 / fp16 (rows may be strided), packed by expert as moe_dispatch does, w
    [G, N, K] of x's type, or [G, K, N] with ``transposed`` (the forward product's weights as they
    are: the gradient of its input), m_sizes [G] int64 -> out [total_M, N] of x's type.  Rows past
    sum(m_sizes) are not written: a freshly allocated ``out`` is zeroed first."""
    b = _binding()
    if out is None:
        M, shape = _moe._shape(x, "x")[0], _stack_shape(w, "w")
        out = _moe._new(stream, (M, shape[2 if transposed else 1]), x.dtype, zero=True)
    s = b.grouped_mm(x, w, m_sizes, transposed, out, _moe._raw(stream))
    if s:
        raise _fx.MslkbError(s, "grouped_mm")
    return out


def grouped_mm_weight_grad(dy, x, m_sizes, *, add=None, dtype=None, out=None, stream=None):
    """dw[g] = add[g] + dy_g^T . x_g over expert g's rows: the gradient of grouped_mm's weights.

    dy [total_M, N], x [total_M, K] bf16 / fp16 (rows may be strided), m_sizes [G] int64 -> dw
    [G, N, K] in ``dtype`` (fp32, the default, or dy's; that of ``add`` where it is given).  ``add``
    is what was accumulated before and may be ``out`` itself.  Rows past sum(m_sizes) are not used;
    an expert without rows gets ``add``, or zeros."""
    b = _binding()
    if out is None:
        torch = _moe._torch
        N, K = _moe._shape(dy, "dy")[1], _moe._shape(x, "x")[1]
        if not isinstance(m_sizes, torch.Tensor):
            raise TypeError("m_sizes must be a torch.Tensor")
        if dtype is None:
            dtype = torch.float32 if add is None else add.dtype
        if dtype not in (torch.float32, dy.dtype):
            raise TypeError(f"dtype {dtype} is neither float32 nor dy's")
        out = _moe._new(stream, (m_sizes.numel(), N, K), dtype)
    s = b.grouped_mm_weight_grad(dy, x, m_sizes, add, out, _moe._raw(stream))
    if s:
        raise _fx.MslkbError(s, "grouped_mm_weight_grad")
    return out
