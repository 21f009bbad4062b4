"""Operators around the grouped product in a mixture-of-experts block.

    add_rms_norm_quant -> (router's logits) -> route_experts -> moe_dispatch
      -> grouped gate/up product -> swiglu_quant -> grouped down product -> moe_combine

and the gradients of the four.  As in the package itself, ``mslkb_*`` functions mirror the C
entry points (raw integer pointers, status returned) and the others take torch CUDA tensors,
which a small extension (csrc/binding.cpp) checks and passes on; all computation happens in
libmslkb.so and nothing falls back.

The torch forms run on the current stream, or on ``stream`` (a torch stream or a raw
cudaStream_t).  Results go to the tensors of ``out`` where it is given (the tuple that the
call returns, e.g. the previous step's), else to new ones; tensors made here belong to the
stream of the call.  All tensors of a call are on the current device.
"""
from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple

import fp8_rowwise_scaled_gb300 as _fx

MSLKB_BF16, MSLKB_FP16, MSLKB_FP32 = range(3)
MSLKB_SOFTMAX, MSLKB_SIGMOID = range(2)
SCALE_BLOCK = 128
MAX_HIDDEN, MAX_TOPK, MAX_EXPERTS = 32768, 32, 1024


def declare(L: ctypes.CDLL) -> ctypes.CDLL:
    """Argument and result types of this module's entry points on a loaded library."""
    p, i64, i32, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double
    for name, args in {
            "mslkb_add_rms_norm_quant": [p] * 8 + [i64] * 4 + [f64, i32, i32, i32, p],
            "mslkb_add_rms_norm_quant_backward": [p] * 8 + [i64] * 3 + [i32, i32, p],
            "mslkb_route_experts": [p] * 4 + [i64] * 4 + [i32, i64, i64, i32, i32, f64, i32, p],
            "mslkb_route_experts_backward": [p] * 4 + [i64] * 4 + [i32, i32, f64, i32, p],
            "mslkb_moe_dispatch": [p] * 7 + [i64] * 5 + [p],
            "mslkb_moe_combine": [p] * 4 + [i64] * 4 + [i32, p],
            "mslkb_moe_combine_backward": [p] * 6 + [i64] * 4 + [i32, p],
            "mslkb_swiglu_quant": [p] * 5 + [i64] * 3 + [i32, i32, p],
            "mslkb_swiglu_quant_backward": [p] * 4 + [i64] * 2 + [i32, p]}.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    L.mslkb_add_rms_norm_quant_backward_workspace_bytes.argtypes = [i64, i64]
    L.mslkb_add_rms_norm_quant_backward_workspace_bytes.restype = i64
    return L


# ---------------------------------------------------------------------------------------
# raw C entry points (integer pointers, None for NULL)
# ---------------------------------------------------------------------------------------
def mslkb_add_rms_norm_quant(x, residual, weight, q, scale, residual_out, y, rstd, T, H, ldx, ldr,
                             eps, dtype, weight_fp32=0, groupwise=0, stream=0) -> int:
    return _fx.lib().mslkb_add_rms_norm_quant(x, residual, weight, q, scale, residual_out, y,
                                              rstd, T, H, ldx, ldr, eps, dtype, weight_fp32,
                                              groupwise, stream)


def mslkb_add_rms_norm_quant_backward_workspace_bytes(T, H) -> int:
    return _fx.lib().mslkb_add_rms_norm_quant_backward_workspace_bytes(T, H)


def mslkb_add_rms_norm_quant_backward(dy, h, weight, rstd, dresidual, dx, dweight, workspace,
                                      workspace_bytes, T, H, dtype, weight_fp32=0,
                                      stream=0) -> int:
    return _fx.lib().mslkb_add_rms_norm_quant_backward(dy, h, weight, rstd, dresidual, dx,
                                                       dweight, workspace, workspace_bytes, T, H,
                                                       dtype, weight_fp32, stream)


def mslkb_route_experts(logits, bias, ids, weights, T, E, ld, top_k, score, num_groups,
                        topk_groups, group_top, renormalize, scale, dtype, stream=0) -> int:
    return _fx.lib().mslkb_route_experts(logits, bias, ids, weights, T, E, ld, top_k, score,
                                         num_groups, topk_groups, group_top, renormalize, scale,
                                         dtype, stream)


def mslkb_route_experts_backward(dweights, logits, ids, dlogits, T, E, ld, top_k, score,
                                 renormalize, scale, dtype, stream=0) -> int:
    return _fx.lib().mslkb_route_experts_backward(dweights, logits, ids, dlogits, T, E, ld, top_k,
                                                  score, renormalize, scale, dtype, stream)


def mslkb_moe_dispatch(x, x_scale, ids, x_out, scale_out, m_sizes, dest, T, top_k, E, row_bytes,
                       scale_cols, stream=0) -> int:
    return _fx.lib().mslkb_moe_dispatch(x, x_scale, ids, x_out, scale_out, m_sizes, dest, T,
                                        top_k, E, row_bytes, scale_cols, stream)


def mslkb_moe_combine(rows, dest, weights, out, T, top_k, H, R, dtype, stream=0) -> int:
    return _fx.lib().mslkb_moe_combine(rows, dest, weights, out, T, top_k, H, R, dtype, stream)


def mslkb_moe_combine_backward(dout, rows, dest, weights, drows, dweights, T, top_k, H, R, dtype,
                               stream=0) -> int:
    return _fx.lib().mslkb_moe_combine_backward(dout, rows, dest, weights, drows, dweights, T,
                                                top_k, H, R, dtype, stream)


def mslkb_swiglu_quant(x, q, scale, saved, saved_scale, R, W, ldx, dtype, groupwise=0,
                       stream=0) -> int:
    return _fx.lib().mslkb_swiglu_quant(x, q, scale, saved, saved_scale, R, W, ldx, dtype,
                                        groupwise, stream)


def mslkb_swiglu_quant_backward(dy, saved, saved_scale, dx, R, W, dtype, stream=0) -> int:
    return _fx.lib().mslkb_swiglu_quant_backward(dy, saved, saved_scale, dx, R, W, dtype, stream)


# ---------------------------------------------------------------------------------------
# torch front end
# ---------------------------------------------------------------------------------------
class NormQuant(NamedTuple):
    """q e4m3 [T, H]; scale fp32 [T] or [T, H/128]; residual, y (x's type) and rstd (fp32 [T])
    where asked for, else None."""
    q: object
    scale: object
    residual: object
    y: object
    rstd: object


class Routing(NamedTuple):
    """ids int32 [T, top_k] (-1: no expert left); weights fp32 [T, top_k]."""
    ids: object
    weights: object


class Dispatch(NamedTuple):
    """x [T*top_k, H] and x_scale packed by expert, m_sizes int64 [E], dest int32 [T, top_k]
    (row of each choice, -1: not here)."""
    x: object
    x_scale: object
    m_sizes: object
    dest: object


class SwigluQuant(NamedTuple):
    """q e4m3 [R, W]; scale fp32 [R] or [R, W/128]; saved e4m3 [R, 2W] and saved_scale fp32
    [R, 2W/128], the checkpoint, or None."""
    q: object
    scale: object
    saved: object
    saved_scale: object


_torch = _b = None
_setup_lock = threading.Lock()


def _setup():
    """Loads the extension that checks and passes tensors (csrc/binding.cpp), and torch, which
    the package imports only when it is used.  `_b` is set last: a thread that finds it set has
    everything."""
    global _torch, _b
    with _setup_lock:
        if _b is not None:
            return
        _fx.lib()
        import torch
        from . import build
        binding = build.load_binding()
        _torch = torch
        _b = binding


def _stream(stream):
    """`stream` as a torch stream."""
    return stream if hasattr(stream, "cuda_stream") else _torch.cuda.ExternalStream(int(stream))


def _new(stream, shape, dtype, zero=False):
    """A tensor on the current device that belongs to the stream of the call."""
    make = _torch.zeros if zero else _torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device="cuda")
    with _torch.cuda.stream(_stream(stream)):
        return make(shape, dtype=dtype, device="cuda")


_NO_COLUMNS = -1   # of csrc/binding.cpp: nothing was written


def _fill(stream, *pairs):
    """The results per row of rows without columns: (tensor or None, value)."""
    with _torch.cuda.stream(None if stream is None else _stream(stream)):
        for t, value in pairs:
            if t is not None:
                t.fill_(value)


def _raw(stream):
    return None if stream is None else _fx._stream_ptr(stream)


def _scale_shape(rows, cols, groupwise):
    if not groupwise:
        return (rows,)
    if cols % SCALE_BLOCK:
        raise ValueError(f"groupwise scales need rows of whole blocks of {SCALE_BLOCK}")
    return (rows, cols // SCALE_BLOCK)


def _shape(t, name):
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dims, got {t.dim()}")
    return t.shape


def _count(n, most, name):
    """A number that results are allocated by."""
    if not 0 <= n <= most:
        raise ValueError(f"{name} must be from 0 to {most}, not {n}")
    return n


def add_rms_norm_quant(x, weight, residual=None, *, eps=1e-6, groupwise=False, want_y=False,
                       want_rstd=False, out=None, stream=None):
    """h = x + residual; y = h * (mean(h^2) + eps)^(-1/2) * weight; q, scale = e4m3 of y.

    x, residual [T, H] bf16 / fp16 / fp32 (rows may be strided); weight [H] of x's type or
    fp32 -> NormQuant(q e4m3 [T, H], scale fp32 [T], or [T, H/128] with ``groupwise``,
    residual = h where a residual was given, y with ``want_y``, rstd with ``want_rstd``).
    q and scale are XQ and x_scale of the rowwise or block-scaled products; the residual of
    ``out`` may be ``residual`` itself."""
    if _b is None:
        _setup()
    if out is None:
        T, H = _shape(x, "x")
        f32 = _torch.float32
        out = NormQuant(_new(stream, (T, H), _torch.float8_e4m3fn),
                        _new(stream, _scale_shape(T, H, groupwise), f32),
                        None if residual is None else _new(stream, (T, H), x.dtype),
                        _new(stream, (T, H), x.dtype) if want_y else None,
                        _new(stream, (T,), f32) if want_rstd else None)
    s = _b.add_rms_norm_quant(x, weight, residual, eps, groupwise, want_y, want_rstd, out,
                              _raw(stream))
    if s == _NO_COLUMNS:
        _fill(stream, (out[1], 1.0), (out[4], eps ** -0.5))
    elif s:
        raise _fx.MslkbError(s, "add_rms_norm_quant")
    return out


def add_rms_norm_quant_backward(dy, h, weight, rstd, dresidual=None, *, out=None, stream=None):
    """Gradient of the norm: dy [T, H] (of y; the quantisation passes it through), h the sum
    that was normalised (NormQuant.residual, or x where there was none), rstd [T] fp32,
    dresidual [T, H] the gradient of NormQuant.residual -> (dx [T, H], the gradient of x and
    of residual alike, dweight [H] fp32)."""
    if _b is None:
        _setup()
    if out is None:
        T, H = _shape(dy, "dy")
        out = _new(stream, (T, H), dy.dtype), _new(stream, (H,), _torch.float32)
    s = _b.add_rms_norm_quant_backward(dy, h, weight, rstd, dresidual, out, _raw(stream))
    if s:
        raise _fx.MslkbError(s, "add_rms_norm_quant_backward")
    return out


_SCORES = {"softmax": MSLKB_SOFTMAX, "sigmoid": MSLKB_SIGMOID}


def _score(score):
    v = _SCORES.get(score)
    if v is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', not {score!r}")
    return v


def route_experts(logits, top_k, *, bias=None, score="softmax", num_groups=1, topk_groups=1,
                  group_top=1, renormalize=True, scale=1.0, out=None, stream=None):
    """Each token's top_k experts and their weights from logits [T, E] (bf16 / fp16 / fp32,
    rows may be strided) -> Routing(ids int32 [T, top_k], weights fp32 [T, top_k]).

    Experts are taken by score (softmax or sigmoid of the logits) + ``bias`` (fp32 [E], for
    balance; not in the weights), best first, the lowest index among equals; with
    ``num_groups`` > 1 only from the ``topk_groups`` groups whose ``group_top`` best choices
    sum highest.  weights = scale * score, over the sum of the taken scores if
    ``renormalize``.  Experts with logit -inf are never taken; slots left get id -1, weight 0."""
    if _b is None:
        _setup()
    if out is None:
        shape = (_shape(logits, "logits")[0], _count(top_k, MAX_TOPK, "top_k"))
        out = Routing(_new(stream, shape, _torch.int32), _new(stream, shape, _torch.float32))
    s = _b.route_experts(logits, top_k, bias, _score(score), num_groups, topk_groups, group_top,
                         renormalize, scale, out, _raw(stream))
    if s:
        raise _fx.MslkbError(s, "route_experts")
    return out


def route_experts_backward(dweights, logits, ids, *, score="softmax", renormalize=True,
                           scale=1.0, out=None, stream=None):
    """dlogits [T, E] (logits' type) from dweights fp32 [T, top_k] for the choice ``ids`` of
    route_experts called with the same score, renormalize and scale."""
    if _b is None:
        _setup()
    if out is None:
        out = _new(stream, _shape(logits, "logits"), logits.dtype)
    s = _b.route_experts_backward(dweights, logits, ids, _score(score), renormalize, scale, out,
                                  _raw(stream))
    if s:
        raise _fx.MslkbError(s, "route_experts_backward")
    return out


def moe_dispatch(x, x_scale, ids, num_experts, *, out=None, stream=None):
    """Packs rows by expert for the stacked products: x [T, H] (e4m3 codes, or any type),
    x_scale fp32 [T], [T, S] or None, ids int32 [T, top_k] -> Dispatch(x [T*top_k, H],
    x_scale [T*top_k(, S)], m_sizes int64 [num_experts], dest int32 [T, top_k]).

    Rows are ordered by expert, then by token; choices outside [0, num_experts) are left out
    (dest -1).  Rows past sum(m_sizes) are not written: buffers allocated here are zeroed
    first so that no stale memory is returned there."""
    if _b is None:
        _setup()
    if out is None:
        H, (T, k) = _shape(x, "x")[1], _shape(ids, "ids")
        _count(k, MAX_TOPK, "experts per token")
        _count(num_experts, MAX_EXPERTS, "num_experts")
        if x_scale is not None and not isinstance(x_scale, _torch.Tensor):
            raise TypeError("x_scale must be a torch.Tensor")
        out = Dispatch(_new(stream, (T * k, H), x.dtype, zero=True),
                       None if x_scale is None else
                       _new(stream, (T * k, *x_scale.shape[1:]), _torch.float32, zero=True),
                       _new(stream, (num_experts,), _torch.int64),
                       _new(stream, (T, k), _torch.int32))
    s = _b.moe_dispatch(x, x_scale, ids, num_experts, out, _raw(stream))
    if s:
        raise _fx.MslkbError(s, "moe_dispatch")
    return out


def moe_combine(rows, dest, weights=None, *, out=None, stream=None):
    """out[t] = sum over j of weights[t, j] * rows[dest[t, j]]: rows [R, H] bf16 / fp16 / fp32,
    dest int32 [T, top_k] (outside [0, R): left out), weights fp32 [T, top_k] or None (ones:
    the gradient of moe_dispatch) -> [T, H] of rows' type."""
    if _b is None:
        _setup()
    if out is None:
        out = _new(stream, (_shape(dest, "dest")[0], _shape(rows, "rows")[1]), rows.dtype)
    s = _b.moe_combine(rows, dest, weights, out, _raw(stream))
    if s:
        raise _fx.MslkbError(s, "moe_combine")
    return out


def moe_combine_backward(dout, rows, dest, weights, *, out=None, stream=None):
    """Gradient of moe_combine: dout [T, H] -> (drows [R, H]: weights[t, j] * dout[t] at row
    dest[t, j], dweights fp32 [T, top_k]: dout[t] . rows[dest[t, j]]).  Rows that no choice
    names are not written: a drows allocated here is zeroed first."""
    if _b is None:
        _setup()
    if out is None:
        out = (_new(stream, _shape(rows, "rows"), rows.dtype, zero=True),
               _new(stream, _shape(dest, "dest"), _torch.float32))
    s = _b.moe_combine_backward(dout, rows, dest, weights, out, _raw(stream))
    if s:
        raise _fx.MslkbError(s, "moe_combine_backward")
    return out


def swiglu_quant(x, *, groupwise=False, checkpoint=False, out=None, stream=None):
    """The experts' activation: x [R, 2W] bf16 / fp16 / fp32 (gate and up side by side, rows may
    be strided); a = gate * sigmoid(gate) * up -> SwigluQuant(q e4m3 [R, W], scale fp32 [R] or
    [R, W/128], and with ``checkpoint`` x itself in 8 bits for the gradient: saved e4m3
    [R, 2W], saved_scale fp32 [R, 2W/128])."""
    if _b is None:
        _setup()
    if out is None:
        R, W2 = _shape(x, "x")
        f32, e4m3 = _torch.float32, _torch.float8_e4m3fn
        out = SwigluQuant(
            _new(stream, (R, W2 // 2), e4m3),
            _new(stream, _scale_shape(R, W2 // 2, groupwise), f32),
            _new(stream, (R, W2), e4m3) if checkpoint else None,
            _new(stream, _scale_shape(R, W2, True), f32) if checkpoint else None)
    s = _b.swiglu_quant(x, groupwise, checkpoint, out, _raw(stream))
    if s == _NO_COLUMNS:
        _fill(stream, (out[1], 1.0))
    elif s:
        raise _fx.MslkbError(s, "swiglu_quant")
    return out


def swiglu_quant_backward(dy, saved, saved_scale=None, *, out=None, stream=None):
    """dx [R, 2W] (dy's type) from dy [R, W] and what the forward kept: the checkpoint (e4m3
    [R, 2W] with its scales) or x itself (saved_scale None)."""
    if _b is None:
        _setup()
    if out is None:
        R, W = _shape(dy, "dy")
        out = _new(stream, (R, 2 * W), dy.dtype)
    s = _b.swiglu_quant_backward(dy, saved, saved_scale, out, _raw(stream))
    if s:
        raise _fx.MslkbError(s, "swiglu_quant_backward")
    return out
