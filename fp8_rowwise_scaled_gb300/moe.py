"""Operators around the grouped product in a mixture-of-experts block.

    add_rms_norm_quant -> (router's logits) -> route_experts -> moe_dispatch
      -> grouped gate/up product -> swiglu_quant -> grouped down product -> moe_combine

and the gradients of the four.  As in the package itself, ``mslkb_*`` functions mirror the C
entry points (raw integer pointers, status returned) and the others take torch CUDA tensors;
all computation happens in libmslkb.so and nothing falls back.

The torch forms run on the current stream, or on ``stream`` (a torch stream or a raw
cudaStream_t).  Results go to the tensors of ``out`` where it is given (the tuple that the
call returns, e.g. the previous step's), else to new ones; tensors made here belong to the
stream of the call.  All tensors of a call are on the current device.
"""
from __future__ import annotations

import ctypes
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


_torch = None
_DTYPES = {}            # torch dtype -> mslkb_dtype
_F32 = _I32 = _E4M3 = None
_device = _raw_stream = None


def _setup():
    """Fills the names that need torch, which the package imports only when it is used."""
    global _torch, _F32, _I32, _E4M3, _device, _raw_stream
    import torch
    _DTYPES.update({torch.bfloat16: MSLKB_BF16, torch.float16: MSLKB_FP16,
                    torch.float32: MSLKB_FP32})
    _F32, _I32, _E4M3 = torch.float32, torch.int32, torch.float8_e4m3fn
    # the index of the current device, and its current stream as a cudaStream_t: at a few
    # microseconds per call, torch.cuda.current_stream(i).cuda_stream is 1 of them, this 0.1
    _device = torch._C._cuda_getDevice
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _torch = torch


def _lead(t, name):
    """The mslkb_dtype and device of the tensor that leads a call: on the current device."""
    if _torch is None:
        _setup()
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name}: dtype {t.dtype} is not bfloat16, float16 or float32")
    return d, _on_device(t, name)


def _on_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != _device():
        raise ValueError(f"{name} is on another device than the current one")
    return dev


def _dense(t, name, dtype, shape, dev):
    """Checks a dense tensor of a call; returns its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype is not dtype and not (dtype is _E4M3 and t.dtype is _torch.uint8):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the same device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dtype, shape, dev):
    """Checks an input whose rows may be slices of wider rows; returns (address, elements from
    row to row)."""
    if t.is_contiguous():
        return _dense(t, name, dtype, shape, dev), shape[1]
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the same device")
    if t.stride(1) != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    ld = t.stride(0) if shape[0] > 1 else shape[1]
    if ld < shape[1]:
        raise ValueError(f"{name}: rows must not overlap (stride {ld} < {shape[1]})")
    return t.data_ptr(), ld


def _stream(stream, dev):
    """The cudaStream_t of a call."""
    return _raw_stream(dev) if stream is None else _fx._stream_ptr(stream)


def _new(stream, dev, shape, dtype, zero=False):
    """A tensor that belongs to the stream of the call."""
    make = _torch.zeros if zero else _torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device="cuda")
    s = stream if hasattr(stream, "cuda_stream") else \
        _torch.cuda.ExternalStream(int(stream), device=_torch.device("cuda", dev))
    with _torch.cuda.stream(s):
        return make(shape, dtype=dtype, device="cuda")


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dims, got {t.dim()}")
    return t.shape


def _unpack(out, count):
    if len(out) != count:
        raise ValueError(f"out must hold {count} tensors (None where there is none)")
    return out


def _same(t, name, wanted):
    if (t is not None) != bool(wanted):
        raise ValueError(f"out: {name} must be {'a tensor' if wanted else 'None'}")


def _scale_shape(rows, cols, groupwise):
    if not groupwise:
        return (rows,)
    if cols % SCALE_BLOCK:
        raise ValueError(f"groupwise scales need rows of whole blocks of {SCALE_BLOCK}")
    return (rows, cols // SCALE_BLOCK)


def _call(status, where):
    if status:
        raise _fx.MslkbError(status, where)


def _weight(weight, dtype, H, dev):
    """Address of a norm weight of x's type or fp32, and whether it is fp32 beside another x."""
    fp32 = weight.dtype is _F32 and dtype is not _F32
    return _dense(weight, "weight", _F32 if fp32 else dtype, (H,), dev), 1 if fp32 else 0


def add_rms_norm_quant(x, weight, residual=None, *, eps=1e-6, groupwise=False, want_y=False,
                       want_rstd=False, out=None, stream=None):
    """h = x + residual; y = h * (mean(h^2) + eps)^(-1/2) * weight; q, scale = e4m3 of y.

    x, residual [T, H] bf16 / fp16 / fp32 (rows may be strided); weight [H] of x's type or
    fp32 -> NormQuant(q e4m3 [T, H], scale fp32 [T], or [T, H/128] with ``groupwise``,
    residual = h where a residual was given, y with ``want_y``, rstd with ``want_rstd``).
    q and scale are XQ and x_scale of the rowwise or block-scaled products; the residual of
    ``out`` may be ``residual`` itself."""
    dt, dev = _lead(x, "x")
    shape = T, H = _matrix(x, "x")
    xt = x.dtype
    xp, ldx = _rows(x, "x", xt, shape, dev)
    rp, ldr = (None, H) if residual is None else _rows(residual, "residual", xt, shape, dev)
    wp, fp32 = _weight(weight, xt, H, dev)
    ss = _scale_shape(T, H, groupwise)
    if out is None:
        q, scale = _new(stream, dev, shape, _E4M3), _new(stream, dev, ss, _F32)
        res = None if residual is None else _new(stream, dev, shape, xt)
        y = _new(stream, dev, shape, xt) if want_y else None
        rstd = _new(stream, dev, (T,), _F32) if want_rstd else None
        out = NormQuant(q, scale, res, y, rstd)
    else:
        q, scale, res, y, rstd = _unpack(out, 5)
        _same(res, "residual", residual is not None)
        _same(y, "y", want_y)
        _same(rstd, "rstd", want_rstd)
    _call(_fx.lib().mslkb_add_rms_norm_quant(
        xp, rp, wp, _dense(q, "q", _E4M3, shape, dev), _dense(scale, "scale", _F32, ss, dev),
        None if res is None else _dense(res, "residual (out)", xt, shape, dev),
        None if y is None else _dense(y, "y", xt, shape, dev),
        None if rstd is None else _dense(rstd, "rstd", _F32, (T,), dev),
        T, H, ldx, ldr, eps, dt, fp32, 1 if groupwise else 0, _stream(stream, dev)),
        "add_rms_norm_quant")
    return out


def add_rms_norm_quant_backward(dy, h, weight, rstd, dresidual=None, *, out=None, stream=None):
    """Gradient of the norm: dy [T, H] (of y; the quantisation passes it through), h the sum
    that was normalised (NormQuant.residual, or x where there was none), rstd [T] fp32,
    dresidual [T, H] the gradient of NormQuant.residual -> (dx [T, H], the gradient of x and
    of residual alike, dweight [H] fp32)."""
    dt, dev = _lead(dy, "dy")
    shape = T, H = _matrix(dy, "dy")
    xt = dy.dtype
    wp, fp32 = _weight(weight, xt, H, dev)
    if out is None:
        out = dx, dw = _new(stream, dev, shape, xt), _new(stream, dev, (H,), _F32)
    else:
        dx, dw = _unpack(out, 2)
    L = _fx.lib()
    need = L.mslkb_add_rms_norm_quant_backward_workspace_bytes(T, H)
    ws = _new(stream, dev, (need,), _torch.uint8)
    _call(L.mslkb_add_rms_norm_quant_backward(
        _dense(dy, "dy", xt, shape, dev), _dense(h, "h", xt, shape, dev), wp,
        _dense(rstd, "rstd", _F32, (T,), dev),
        None if dresidual is None else _dense(dresidual, "dresidual", xt, shape, dev),
        _dense(dx, "dx", xt, shape, dev), _dense(dw, "dweight", _F32, (H,), dev),
        ws.data_ptr(), need, T, H, dt, fp32, _stream(stream, dev)),
        "add_rms_norm_quant_backward")
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
    dt, dev = _lead(logits, "logits")
    T, E = _matrix(logits, "logits")
    lp, ld = _rows(logits, "logits", logits.dtype, (T, E), dev)
    kind = _score(score)
    shape = (T, top_k)
    if out is None:
        out = Routing(_new(stream, dev, shape, _I32), _new(stream, dev, shape, _F32))
    ids, weights = _unpack(out, 2)
    _call(_fx.lib().mslkb_route_experts(
        lp, None if bias is None else _dense(bias, "bias", _F32, (E,), dev),
        _dense(ids, "ids", _I32, shape, dev), _dense(weights, "weights", _F32, shape, dev),
        T, E, ld, top_k, kind, num_groups, topk_groups, group_top, 1 if renormalize else 0,
        scale, dt, _stream(stream, dev)), "route_experts")
    return out


def route_experts_backward(dweights, logits, ids, *, score="softmax", renormalize=True,
                           scale=1.0, out=None, stream=None):
    """dlogits [T, E] (logits' type) from dweights fp32 [T, top_k] for the choice ``ids`` of
    route_experts called with the same score, renormalize and scale."""
    dt, dev = _lead(logits, "logits")
    T, E = _matrix(logits, "logits")
    lp, ld = _rows(logits, "logits", logits.dtype, (T, E), dev)
    shape = _matrix(ids, "ids")
    if shape[0] != T:
        raise ValueError("ids and logits disagree on the number of tokens")
    if out is None:
        out = _new(stream, dev, (T, E), logits.dtype)
    _call(_fx.lib().mslkb_route_experts_backward(
        _dense(dweights, "dweights", _F32, shape, dev), lp, _dense(ids, "ids", _I32, shape, dev),
        _dense(out, "out", logits.dtype, (T, E), dev), T, E, ld, shape[1], _score(score),
        1 if renormalize else 0, scale, dt, _stream(stream, dev)), "route_experts_backward")
    return out


def moe_dispatch(x, x_scale, ids, num_experts, *, out=None, stream=None):
    """Packs rows by expert for the stacked products: x [T, H] (e4m3 codes, or any type),
    x_scale fp32 [T], [T, S] or None, ids int32 [T, top_k] -> Dispatch(x [T*top_k, H],
    x_scale [T*top_k(, S)], m_sizes int64 [num_experts], dest int32 [T, top_k]).

    Rows are ordered by expert, then by token; choices outside [0, num_experts) are left out
    (dest -1).  Rows past sum(m_sizes) are not written: buffers allocated here are zeroed
    first so that no stale memory is returned there."""
    if _torch is None:
        _setup()
    dev = _on_device(x, "x")
    T, H = _matrix(x, "x")
    k = _matrix(ids, "ids")[1]
    xp = _dense(x, "x", x.dtype, (T, H), dev)
    ip = _dense(ids, "ids", _I32, (T, k), dev)
    sp, cols, tail = None, 0, ()
    if x_scale is not None:
        if x_scale.dim() not in (1, 2):
            raise ValueError(f"x_scale: expected 1 or 2 dims, got {x_scale.dim()}")
        tail = tuple(x_scale.shape[1:])
        cols = tail[0] if tail else 1
        sp = _dense(x_scale, "x_scale", _F32, (T, *tail), dev)
    N = T * k
    if out is None:
        out = Dispatch(_new(stream, dev, (N, H), x.dtype, zero=True),
                       None if x_scale is None else _new(stream, dev, (N, *tail), _F32, zero=True),
                       _new(stream, dev, (num_experts,), _torch.int64),
                       _new(stream, dev, (T, k), _I32))
    xo, so, m_sizes, dest = _unpack(out, 4)
    _same(so, "x_scale", x_scale is not None)
    _call(_fx.lib().mslkb_moe_dispatch(
        xp, sp, ip, _dense(xo, "x (out)", x.dtype, (N, H), dev),
        None if so is None else _dense(so, "x_scale (out)", _F32, (N, *tail), dev),
        _dense(m_sizes, "m_sizes", _torch.int64, (num_experts,), dev),
        _dense(dest, "dest", _I32, (T, k), dev), T, k, num_experts, H * x.element_size(), cols,
        _stream(stream, dev)), "moe_dispatch")
    return out


def moe_combine(rows, dest, weights=None, *, out=None, stream=None):
    """out[t] = sum over j of weights[t, j] * rows[dest[t, j]]: rows [R, H] bf16 / fp16 / fp32,
    dest int32 [T, top_k] (outside [0, R): left out), weights fp32 [T, top_k] or None (ones:
    the gradient of moe_dispatch) -> [T, H] of rows' type."""
    dt, dev = _lead(rows, "rows")
    shape = R, H = _matrix(rows, "rows")
    choices = T, k = _matrix(dest, "dest")
    if out is None:
        out = _new(stream, dev, (T, H), rows.dtype)
    _call(_fx.lib().mslkb_moe_combine(
        _dense(rows, "rows", rows.dtype, shape, dev), _dense(dest, "dest", _I32, choices, dev),
        None if weights is None else _dense(weights, "weights", _F32, choices, dev),
        _dense(out, "out", rows.dtype, (T, H), dev), T, k, H, R, dt, _stream(stream, dev)),
        "moe_combine")
    return out


def moe_combine_backward(dout, rows, dest, weights, *, out=None, stream=None):
    """Gradient of moe_combine: dout [T, H] -> (drows [R, H]: weights[t, j] * dout[t] at row
    dest[t, j], dweights fp32 [T, top_k]: dout[t] . rows[dest[t, j]]).  Rows that no choice
    names are not written: a drows allocated here is zeroed first."""
    dt, dev = _lead(dout, "dout")
    T, H = _matrix(dout, "dout")
    R = _matrix(rows, "rows")[0]
    k = _matrix(dest, "dest")[1]
    xt = dout.dtype
    if out is None:
        out = (_new(stream, dev, (R, H), xt, zero=True), _new(stream, dev, (T, k), _F32))
    drows, dw = _unpack(out, 2)
    _call(_fx.lib().mslkb_moe_combine_backward(
        _dense(dout, "dout", xt, (T, H), dev), _dense(rows, "rows", xt, (R, H), dev),
        _dense(dest, "dest", _I32, (T, k), dev), _dense(weights, "weights", _F32, (T, k), dev),
        _dense(drows, "drows", xt, (R, H), dev), _dense(dw, "dweights", _F32, (T, k), dev),
        T, k, H, R, dt, _stream(stream, dev)), "moe_combine_backward")
    return out


def swiglu_quant(x, *, groupwise=False, checkpoint=False, out=None, stream=None):
    """The experts' activation: x [R, 2W] bf16 / fp16 / fp32 (gate and up side by side, rows may
    be strided); a = gate * sigmoid(gate) * up -> SwigluQuant(q e4m3 [R, W], scale fp32 [R] or
    [R, W/128], and with ``checkpoint`` x itself in 8 bits for the gradient: saved e4m3
    [R, 2W], saved_scale fp32 [R, 2W/128])."""
    dt, dev = _lead(x, "x")
    R, W2 = _matrix(x, "x")
    if W2 % 2:
        raise ValueError("x holds gate and up side by side: an even number of columns")
    W = W2 // 2
    xp, ldx = _rows(x, "x", x.dtype, (R, W2), dev)
    ss = _scale_shape(R, W, groupwise)
    kept = (R, 2 * _scale_shape(R, W, True)[1]) if checkpoint else None
    if out is None:
        out = SwigluQuant(_new(stream, dev, (R, W), _E4M3), _new(stream, dev, ss, _F32),
                          _new(stream, dev, (R, W2), _E4M3) if checkpoint else None,
                          _new(stream, dev, kept, _F32) if checkpoint else None)
    q, scale, saved, saved_scale = _unpack(out, 4)
    _same(saved, "saved", checkpoint)
    _same(saved_scale, "saved_scale", checkpoint)
    _call(_fx.lib().mslkb_swiglu_quant(
        xp, _dense(q, "q", _E4M3, (R, W), dev), _dense(scale, "scale", _F32, ss, dev),
        None if saved is None else _dense(saved, "saved", _E4M3, (R, W2), dev),
        None if saved is None else _dense(saved_scale, "saved_scale", _F32, kept, dev),
        R, W, ldx, dt, 1 if groupwise else 0, _stream(stream, dev)), "swiglu_quant")
    return out


def swiglu_quant_backward(dy, saved, saved_scale=None, *, out=None, stream=None):
    """dx [R, 2W] (dy's type) from dy [R, W] and what the forward kept: the checkpoint (e4m3
    [R, 2W] with its scales) or x itself (saved_scale None)."""
    dt, dev = _lead(dy, "dy")
    R, W = _matrix(dy, "dy")
    xt = dy.dtype
    if out is None:
        out = _new(stream, dev, (R, 2 * W), xt)
    if saved_scale is None:
        kp, sp = _dense(saved, "saved", xt, (R, 2 * W), dev), None
    else:
        kp = _dense(saved, "saved", _E4M3, (R, 2 * W), dev)
        sp = _dense(saved_scale, "saved_scale", _F32, (R, 2 * _scale_shape(R, W, True)[1]), dev)
    _call(_fx.lib().mslkb_swiglu_quant_backward(
        _dense(dy, "dy", xt, (R, W), dev), kp, sp, _dense(out, "out", xt, (R, 2 * W), dev),
        R, W, dt, _stream(stream, dev)), "swiglu_quant_backward")
    return out
