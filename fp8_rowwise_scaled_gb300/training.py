"""Operators for training the experts: their products in 16 bits, forward and backward, and what
follows the backward pass.

    grouped_mm(x, w) -> ... -> grouped_mm(dy, w, transposed=True)     the input's gradient
                               grouped_mm_weight_grad(dy, x)          the weights' gradient
                            -> clip_grad_norm(all gradients)          (or grad_norm alone)

As in moe.py, whose conventions hold here too: ``mslkb_*`` functions mirror the C entry points,
the others take torch CUDA tensors, run on the current stream or on ``stream``, and put their
results into ``out`` where it is given.

As there, autograd sees none of it: a result of inputs that require a gradient is detached, and
what is written in place (``out`` over a gradient, or over ``add``) does not raise the tensor's
version.  A backward pass calls the gradients' functions itself.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import fp8_rowwise_scaled_gb300 as _fx

from . import moe as _moe

MSLKB_NORM_2, MSLKB_NORM_INF = range(2)
MAX_TENSORS = 65536


def declare(L: ctypes.CDLL) -> ctypes.CDLL:
    """Argument and result types of this module's entry points on a loaded library."""
    p, i64, i32, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double
    for name, args in {
            "mslkb_grouped_mm": [p] * 4 + [i64] * 5 + [i32, i32, p, i64, p],
            "mslkb_grouped_mm_weight_grad": [p] * 5 + [i64] * 6 + [i32, i32, p, i64, p],
            "mslkb_grad_norm": [p] * 3 + [i64, i32, p, p, i64, p],
            "mslkb_clip_grad_norm": [p] * 4 + [i64, i32, f64, f64, p, p, i64, p]}.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    for name, args in {
            "mslkb_grouped_mm_workspace_bytes": [p] * 2 + [i64] * 5 + [i32],
            "mslkb_grouped_mm_weight_grad_workspace_bytes": [p] * 2 + [i64] * 6,
            "mslkb_grad_norm_workspace_bytes": [i64]}.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, i64
    return L


# ---------------------------------------------------------------------------------------
# raw C entry points (integer pointers, None for NULL)
# ---------------------------------------------------------------------------------------
def mslkb_grouped_mm_workspace_bytes(x, w, total_M, G, N, K, ldx, transposed=0) -> int:
    return _fx.lib().mslkb_grouped_mm_workspace_bytes(x, w, total_M, G, N, K, ldx, transposed)


def mslkb_grouped_mm(x, w, m_sizes, out, total_M, G, N, K, ldx, transposed, dtype, workspace=None,
                     workspace_bytes=0, stream=0) -> int:
    return _fx.lib().mslkb_grouped_mm(x, w, m_sizes, out, total_M, G, N, K, ldx, transposed,
                                      dtype, workspace, workspace_bytes, stream)


def mslkb_grouped_mm_weight_grad_workspace_bytes(dy, x, total_M, G, N, K, lddy, ldx) -> int:
    return _fx.lib().mslkb_grouped_mm_weight_grad_workspace_bytes(dy, x, total_M, G, N, K, lddy,
                                                                  ldx)


def mslkb_grouped_mm_weight_grad(dy, x, m_sizes, add, dw, total_M, G, N, K, lddy, ldx, dtype,
                                 dw_fp32=1, workspace=None, workspace_bytes=0, stream=0) -> int:
    return _fx.lib().mslkb_grouped_mm_weight_grad(dy, x, m_sizes, add, dw, total_M, G, N, K, lddy,
                                                  ldx, dtype, dw_fp32, workspace, workspace_bytes,
                                                  stream)


def mslkb_grad_norm_workspace_bytes(count) -> int:
    return _fx.lib().mslkb_grad_norm_workspace_bytes(count)


def mslkb_grad_norm(grads, sizes, dtypes, count, kind, norm, workspace, workspace_bytes,
                    stream=0) -> int:
    """grads, sizes, dtypes: host arrays (ctypes arrays or addresses)."""
    return _fx.lib().mslkb_grad_norm(grads, sizes, dtypes, count, kind, norm, workspace,
                                     workspace_bytes, stream)


def mslkb_clip_grad_norm(grads, outs, sizes, dtypes, count, kind, max_norm, eps, norm, workspace,
                         workspace_bytes, stream=0) -> int:
    return _fx.lib().mslkb_clip_grad_norm(grads, outs, sizes, dtypes, count, kind, max_norm, eps,
                                          norm, workspace, workspace_bytes, stream)


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
    sum(m_sizes) are not written: a freshly allocated ``out`` is zeroed first.  ``out`` must not lie
    over x, w or m_sizes."""
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
    is what was accumulated before and may be ``out`` itself (but must not overlap it otherwise).
    Rows past sum(m_sizes) are not used; an expert without rows gets ``add``, or zeros.  ``out`` must
    not lie over dy, x or m_sizes."""
    b = _binding()
    if out is None:
        torch = _moe._torch
        N, K = _moe._shape(dy, "dy")[1], _moe._shape(x, "x")[1]
        if not isinstance(m_sizes, torch.Tensor):
            raise TypeError("m_sizes must be a torch.Tensor")
        if dtype is None:
            dtype = add.dtype if isinstance(add, torch.Tensor) else torch.float32
        if dtype not in (torch.float32, dy.dtype):
            raise TypeError(f"dtype {dtype} is neither float32 nor dy's")
        out = _moe._new(stream, (m_sizes.numel(), N, K), dtype)
    s = b.grouped_mm_weight_grad(dy, x, m_sizes, add, out, _moe._raw(stream))
    if s:
        raise _fx.MslkbError(s, "grouped_mm_weight_grad")
    return out


class ClippedGrads(NamedTuple):
    """norm fp32 (of the gradients before they were scaled); grads, the scaled gradients."""
    norm: object
    grads: object


def _kind(norm_type):
    if norm_type == 2:
        return MSLKB_NORM_2
    if norm_type == float("inf"):
        return MSLKB_NORM_INF
    raise ValueError(f"norm_type must be 2 or infinity, not {norm_type!r}")


def grad_norm(grads, *, norm_type=2.0, out=None, stream=None):
    """The norm of all gradients taken together as one vector: the square root of the sum of all
    squares, or the largest magnitude (``norm_type`` infinity).

    grads: a list or tuple of dense tensors, each bf16, fp16 or fp32 -> fp32 tensor of one
    element."""
    b = _binding()
    kind = _kind(norm_type)
    if out is None:
        out = _moe._new(stream, (), _moe._torch.float32)
    s = b.grad_norm(grads, kind, out, _moe._raw(stream))
    if s:
        raise _fx.MslkbError(s, "grad_norm")
    return out


def clip_grad_norm(grads, max_norm, *, norm_type=2.0, eps=1e-6, out=None, stream=None):
    """grads * scale -> ClippedGrads(norm, grads): norm is that of grad_norm, scale is 1 where norm +
    eps <= max_norm (always, unless norm is NaN, if max_norm is infinite), else max_norm / (norm +
    eps).

    ``out`` is (norm, tensors of the gradients' types, shapes and strides); the tensors may be the
    gradients themselves, which are then scaled in place (and not written where nothing
    changes), but must not overlap otherwise, nor the norm lie over them.  Without ``out`` new tensors are made."""
    b = _binding()
    kind = _kind(norm_type)
    if out is None:
        torch = _moe._torch
        if not isinstance(grads, (list, tuple)):
            raise TypeError("grads must be a list or tuple of tensors")
        if not all(isinstance(g, torch.Tensor) for g in grads):
            raise TypeError("grads must be a torch.Tensor")
        with torch.cuda.stream(None if stream is None else _moe._stream(stream)):
            out = ClippedGrads(torch.empty((), dtype=torch.float32, device="cuda"),
                               [torch.empty_like(g) for g in grads])
    elif not isinstance(out, tuple) or len(out) != 2:
        raise TypeError("out must be a tuple (norm, tensors)")
    s = b.clip_grad_norm(grads, kind, max_norm, eps, out[0], out[1], _moe._raw(stream))
    if s:
        raise _fx.MslkbError(s, "clip_grad_norm")
    return ClippedGrads(*out)
