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
            "mslkb_moe_dispatch": [p] * 8 + [i64] * 6 + [p],
            "mslkb_moe_combine": [p] * 4 + [i64] * 4 + [i32, p],
            "mslkb_moe_combine_backward": [p] * 6 + [i64] * 4 + [i32, p],
            "mslkb_swiglu_quant": [p] * 5 + [i64] * 3 + [i32, i32, p],
            "mslkb_swiglu_quant_backward": [p] * 4 + [i64] * 2 + [i32, p]}.items():
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    for name, count in (("mslkb_add_rms_norm_quant_backward_workspace_bytes", 2),
                        ("mslkb_moe_dispatch_workspace_bytes", 3)):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = [i64] * count, i64
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


def mslkb_moe_dispatch_workspace_bytes(T, top_k, E) -> int:
    return _fx.lib().mslkb_moe_dispatch_workspace_bytes(T, top_k, E)


def mslkb_moe_dispatch(x, x_scale, ids, x_out, scale_out, m_sizes, dest, workspace,
                       workspace_bytes, T, top_k, E, row_bytes, scale_cols, stream=0) -> int:
    return _fx.lib().mslkb_moe_dispatch(x, x_scale, ids, x_out, scale_out, m_sizes, dest,
                                        workspace, workspace_bytes, T, top_k, E, row_bytes,
                                        scale_cols, stream)


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
_DTYPES = {}       # torch dtype -> mslkb_dtype
_DEVICE = None     # the current device's index


def _setup():
    """Fills the tables that need torch, which the package imports only when it is used."""
    global _torch, _DEVICE
    import torch
    _DTYPES.update({torch.bfloat16: MSLKB_BF16, torch.float16: MSLKB_FP16,
                    torch.float32: MSLKB_FP32})
    _DEVICE = torch.cuda.current_device
    _torch = torch


def _dtype(t, name):
    """The mslkb_dtype of a tensor that leads a call, which must be on the current device."""
    if _torch is None:
        _setup()
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != _DEVICE():
        raise ValueError(f"{name} is on another device than the current one")
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name}: dtype {t.dtype} is not bfloat16, float16 or float32")
    return d


def _dense(t, name, dtype, shape, device):
    """Checks a dense tensor of a call; returns its address."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype and not (dtype is _torch.float8_e4m3fn and t.dtype is _torch.uint8):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on the same device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dtype, shape, device):
    """Checks an input whose rows may be slices of wider rows; returns (address, elements from
    row to row)."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on the same device")
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    if t.stride(1) != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    ld = t.stride(0) if shape[0] > 1 else shape[1]
    if ld < shape[1]:
        raise ValueError(f"{name}: rows must not overlap (stride {ld} < {shape[1]})")
    return t.data_ptr(), ld


class _Stream:
    """The raw stream of a call; `new` makes tensors that belong to it."""

    def __init__(self, stream, device):
        self.stream = stream
        if stream is None:
            self.raw = _torch.cuda.current_stream(device).cuda_stream
        else:
            self.raw = _fx._stream_ptr(stream)

    def new(self, shape, dtype, device, zero=False):
        make = _torch.zeros if zero else _torch.empty
        device = _torch.device("cuda", device)
        if self.stream is None:
            return make(shape, dtype=dtype, device=device)
        s = self.stream if hasattr(self.stream, "cuda_stream") else \
            _torch.cuda.ExternalStream(self.raw, device=device)
        with _torch.cuda.stream(s):
            return make(shape, dtype=dtype, device=device)


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dims, got {t.dim()}")
    return t.shape


def _unpack(out, count):
    if out is None:
        return (None,) * count
    if len(out) != count:
        raise ValueError(f"out must hold {count} tensors (None where there is none)")
    return out


def _scale_shape(rows, cols, groupwise):
    if not groupwise:
        return (rows,)
    if cols % SCALE_BLOCK:
        raise ValueError(f"groupwise scales need rows of whole blocks of {SCALE_BLOCK}")
    return (rows, cols // SCALE_BLOCK)


def _call(status, where):
    if status:
        raise _fx.MslkbError(status, where)


def _weight(weight, dtype, H, device):
    """Address of a norm weight of x's type or fp32, and whether it is fp32 beside another x."""
    fp32 = weight.dtype is _torch.float32 and dtype is not _torch.float32
    return _dense(weight, "weight", _torch.float32 if fp32 else dtype, (H,), device), int(fp32)


def add_rms_norm_quant(x, weight, residual=None, *, eps=1e-6, groupwise=False, want_y=False,
                       want_rstd=False, out=None, stream=None):
    """h = x + residual; y = h * (mean(h^2) + eps)^(-1/2) * weight; q, scale = e4m3 of y.

    x, residual [T, H] bf16 / fp16 / fp32 (rows may be strided); weight [H] of x's type or
    fp32 -> NormQuant(q e4m3 [T, H], scale fp32 [T], or [T, H/128] with ``groupwise``,
    residual = h where a residual was given, y with ``want_y``, rstd with ``want_rstd``).
    q and scale are XQ and x_scale of the rowwise or block-scaled products; the residual of
    ``out`` may be ``residual`` itself."""
    dt = _dtype(x, "x")
    T, H = _matrix(x, "x")
    dev, xt = x.get_device(), x.dtype
    xp, ldx = _rows(x, "x", xt, (T, H), dev)
    rp, ldr = _rows(residual, "residual", xt, (T, H), dev) if residual is not None else (None, H)
    wp, fp32 = _weight(weight, xt, H, dev)
    ss = _scale_shape(T, H, groupwise)
    s = _Stream(stream, dev)
    q, scale, res, y, rstd = _unpack(out, 5)
    if out is None:
        q, scale = s.new((T, H), _torch.float8_e4m3fn, dev), s.new(ss, _torch.float32, dev)
        res = s.new((T, H), xt, dev) if residual is not None else None
        y = s.new((T, H), xt, dev) if want_y else None
        rstd = s.new((T,), _torch.float32, dev) if want_rstd else None
        out = NormQuant(q, scale, res, y, rstd)
    for t, name, wanted in ((res, "residual", residual is not None), (y, "y", want_y),
                            (rstd, "rstd", want_rstd)):
        if (t is not None) != bool(wanted):
            raise ValueError(f"out: {name} must be {'a tensor' if wanted else 'None'}")
    _call(_fx.lib().mslkb_add_rms_norm_quant(
        xp, rp, wp, _dense(q, "q", _torch.float8_e4m3fn, (T, H), dev),
        _dense(scale, "scale", _torch.float32, ss, dev),
        None if res is None else _dense(res, "residual (out)", xt, (T, H), dev),
        None if y is None else _dense(y, "y", xt, (T, H), dev),
        None if rstd is None else _dense(rstd, "rstd", _torch.float32, (T,), dev),
        T, H, ldx, ldr, eps, dt, fp32, int(bool(groupwise)), s.raw), "add_rms_norm_quant")
    return out


def add_rms_norm_quant_backward(dy, h, weight, rstd, dresidual=None, *, out=None, stream=None):
    """Gradient of the norm: dy [T, H] (of y; the quantisation passes it through), h the sum
    that was normalised (NormQuant.residual, or x where there was none), rstd [T] fp32,
    dresidual [T, H] the gradient of NormQuant.residual -> (dx [T, H], the gradient of x and
    of residual alike, dweight [H] fp32)."""
    dt = _dtype(dy, "dy")
    T, H = _matrix(dy, "dy")
    dev, xt = dy.get_device(), dy.dtype
    wp, fp32 = _weight(weight, xt, H, dev)
    s = _Stream(stream, dev)
    dx, dw = _unpack(out, 2)
    if out is None:
        out = dx, dw = s.new((T, H), xt, dev), s.new((H,), _torch.float32, dev)
    L = _fx.lib()
    need = L.mslkb_add_rms_norm_quant_backward_workspace_bytes(T, H)
    ws = s.new((need,), _torch.uint8, dev)
    _call(L.mslkb_add_rms_norm_quant_backward(
        _dense(dy, "dy", xt, (T, H), dev), _dense(h, "h", xt, (T, H), dev), wp,
        _dense(rstd, "rstd", _torch.float32, (T,), dev),
        None if dresidual is None else _dense(dresidual, "dresidual", xt, (T, H), dev),
        _dense(dx, "dx", xt, (T, H), dev), _dense(dw, "dweight", _torch.float32, (H,), dev),
        ws.data_ptr(), need, T, H, dt, fp32, s.raw), "add_rms_norm_quant_backward")
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
    dt = _dtype(logits, "logits")
    T, E = _matrix(logits, "logits")
    dev = logits.get_device()
    lp, ld = _rows(logits, "logits", logits.dtype, (T, E), dev)
    kind = _score(score)
    s = _Stream(stream, dev)
    shape = (T, top_k)
    ids, weights = _unpack(out, 2)
    if out is None:
        out = ids, weights = Routing(s.new(shape, _torch.int32, dev),
                                     s.new(shape, _torch.float32, dev))
    _call(_fx.lib().mslkb_route_experts(
        lp, None if bias is None else _dense(bias, "bias", _torch.float32, (E,), dev),
        _dense(ids, "ids", _torch.int32, shape, dev),
        _dense(weights, "weights", _torch.float32, shape, dev), T, E, ld, top_k, kind,
        num_groups, topk_groups, group_top, int(bool(renormalize)), scale, dt, s.raw),
        "route_experts")
    return out


def route_experts_backward(dweights, logits, ids, *, score="softmax", renormalize=True,
                           scale=1.0, out=None, stream=None):
    """dlogits [T, E] (logits' type) from dweights fp32 [T, top_k] for the choice ``ids`` of
    route_experts called with the same score, renormalize and scale."""
    dt = _dtype(logits, "logits")
    T, E = _matrix(logits, "logits")
    dev = logits.get_device()
    lp, ld = _rows(logits, "logits", logits.dtype, (T, E), dev)
    shape = _matrix(ids, "ids")
    if shape[0] != T:
        raise ValueError("ids and logits disagree on the number of tokens")
    s = _Stream(stream, dev)
    if out is None:
        out = s.new((T, E), logits.dtype, dev)
    _call(_fx.lib().mslkb_route_experts_backward(
        _dense(dweights, "dweights", _torch.float32, shape, dev), lp,
        _dense(ids, "ids", _torch.int32, shape, dev),
        _dense(out, "out", logits.dtype, (T, E), dev), T, E, ld, shape[1], _score(score),
        int(bool(renormalize)), scale, dt, s.raw), "route_experts_backward")
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
    T, H = _matrix(x, "x")
    dev = x.get_device()
    if not x.is_cuda or dev != _DEVICE():
        raise ValueError("x must be a CUDA tensor on the current device")
    k = _matrix(ids, "ids")[1]
    xp = _dense(x, "x", x.dtype, (T, H), dev)
    ip = _dense(ids, "ids", _torch.int32, (T, k), dev)
    sp, cols, tail = None, 0, ()
    if x_scale is not None:
        if x_scale.dim() not in (1, 2):
            raise ValueError(f"x_scale: expected 1 or 2 dims, got {x_scale.dim()}")
        tail = tuple(x_scale.shape[1:])
        cols = tail[0] if tail else 1
        sp = _dense(x_scale, "x_scale", _torch.float32, (T, *tail), dev)
    s = _Stream(stream, dev)
    xo, so, m_sizes, dest = _unpack(out, 4)
    if out is None:
        xo = s.new((T * k, H), x.dtype, dev, zero=True)
        so = s.new((T * k, *tail), _torch.float32, dev, zero=True) if cols else None
        m_sizes = s.new((num_experts,), _torch.int64, dev)
        dest = s.new((T, k), _torch.int32, dev)
        out = Dispatch(xo, so, m_sizes, dest)
    elif (so is None) != (x_scale is None):
        raise ValueError("out: x_scale must be there exactly where the input has one")
    L = _fx.lib()
    need = L.mslkb_moe_dispatch_workspace_bytes(T, k, num_experts)
    ws = s.new((need,), _torch.uint8, dev) if need else None
    _call(L.mslkb_moe_dispatch(
        xp, sp, ip, _dense(xo, "x (out)", x.dtype, (T * k, H), dev),
        None if so is None else _dense(so, "x_scale (out)", _torch.float32, (T * k, *tail), dev),
        _dense(m_sizes, "m_sizes", _torch.int64, (num_experts,), dev),
        _dense(dest, "dest", _torch.int32, (T, k), dev), None if ws is None else ws.data_ptr(),
        need, T, k, num_experts, H * x.element_size(), cols, s.raw), "moe_dispatch")
    return out


def moe_combine(rows, dest, weights=None, *, out=None, stream=None):
    """out[t] = sum over j of weights[t, j] * rows[dest[t, j]]: rows [R, H] bf16 / fp16 / fp32,
    dest int32 [T, top_k] (outside [0, R): left out), weights fp32 [T, top_k] or None (ones:
    the gradient of moe_dispatch) -> [T, H] of rows' type."""
    dt = _dtype(rows, "rows")
    R, H = _matrix(rows, "rows")
    dev = rows.get_device()
    T, k = _matrix(dest, "dest")
    s = _Stream(stream, dev)
    if out is None:
        out = s.new((T, H), rows.dtype, dev)
    _call(_fx.lib().mslkb_moe_combine(
        _dense(rows, "rows", rows.dtype, (R, H), dev),
        _dense(dest, "dest", _torch.int32, (T, k), dev),
        None if weights is None else _dense(weights, "weights", _torch.float32, (T, k), dev),
        _dense(out, "out", rows.dtype, (T, H), dev), T, k, H, R, dt, s.raw), "moe_combine")
    return out


def moe_combine_backward(dout, rows, dest, weights, *, out=None, stream=None):
    """Gradient of moe_combine: dout [T, H] -> (drows [R, H]: weights[t, j] * dout[t] at row
    dest[t, j], dweights fp32 [T, top_k]: dout[t] . rows[dest[t, j]]).  Rows that no choice
    names are not written: a drows allocated here is zeroed first."""
    dt = _dtype(dout, "dout")
    T, H = _matrix(dout, "dout")
    dev = dout.get_device()
    R = _matrix(rows, "rows")[0]
    k = _matrix(dest, "dest")[1]
    s = _Stream(stream, dev)
    drows, dw = _unpack(out, 2)
    if out is None:
        out = drows, dw = (s.new((R, H), dout.dtype, dev, zero=True),
                           s.new((T, k), _torch.float32, dev))
    _call(_fx.lib().mslkb_moe_combine_backward(
        _dense(dout, "dout", dout.dtype, (T, H), dev),
        _dense(rows, "rows", dout.dtype, (R, H), dev),
        _dense(dest, "dest", _torch.int32, (T, k), dev),
        _dense(weights, "weights", _torch.float32, (T, k), dev),
        _dense(drows, "drows", dout.dtype, (R, H), dev),
        _dense(dw, "dweights", _torch.float32, (T, k), dev), T, k, H, R, dt, s.raw),
        "moe_combine_backward")
    return out


def swiglu_quant(x, *, groupwise=False, checkpoint=False, out=None, stream=None):
    """The experts' activation: x [R, 2W] bf16 / fp16 / fp32 (gate and up side by side, rows may
    be strided); a = gate * sigmoid(gate) * up -> SwigluQuant(q e4m3 [R, W], scale fp32 [R] or
    [R, W/128], and with ``checkpoint`` x itself in 8 bits for the gradient: saved e4m3
    [R, 2W], saved_scale fp32 [R, 2W/128])."""
    dt = _dtype(x, "x")
    R, W2 = _matrix(x, "x")
    if W2 % 2:
        raise ValueError("x holds gate and up side by side: an even number of columns")
    W, dev = W2 // 2, x.get_device()
    xp, ldx = _rows(x, "x", x.dtype, (R, W2), dev)
    ss = _scale_shape(R, W, groupwise)
    kept = _scale_shape(R, W, True) if checkpoint else None
    s = _Stream(stream, dev)
    e4m3, f32 = _torch.float8_e4m3fn, _torch.float32
    q, scale, saved, saved_scale = _unpack(out, 4)
    if out is None:
        q, scale = s.new((R, W), e4m3, dev), s.new(ss, f32, dev)
        if checkpoint:
            saved, saved_scale = s.new((R, W2), e4m3, dev), s.new((R, 2 * kept[1]), f32, dev)
        out = SwigluQuant(q, scale, saved, saved_scale)
    if (saved is not None) != bool(checkpoint) or (saved_scale is not None) != bool(checkpoint):
        raise ValueError("out: saved and saved_scale must be there exactly with checkpoint")
    _call(_fx.lib().mslkb_swiglu_quant(
        xp, _dense(q, "q", e4m3, (R, W), dev), _dense(scale, "scale", f32, ss, dev),
        None if saved is None else _dense(saved, "saved", e4m3, (R, W2), dev),
        None if saved is None else _dense(saved_scale, "saved_scale", f32, (R, 2 * kept[1]), dev),
        R, W, ldx, dt, int(bool(groupwise)), s.raw), "swiglu_quant")
    return out


def swiglu_quant_backward(dy, saved, saved_scale=None, *, out=None, stream=None):
    """dx [R, 2W] (dy's type) from dy [R, W] and what the forward kept: the checkpoint (e4m3
    [R, 2W] with its scales) or x itself (saved_scale None)."""
    dt = _dtype(dy, "dy")
    R, W = _matrix(dy, "dy")
    dev = dy.get_device()
    s = _Stream(stream, dev)
    if out is None:
        out = s.new((R, 2 * W), dy.dtype, dev)
    if saved_scale is None:
        kp, sp = _dense(saved, "saved", dy.dtype, (R, 2 * W), dev), None
    else:
        kp = _dense(saved, "saved", _torch.float8_e4m3fn, (R, 2 * W), dev)
        sp = _dense(saved_scale, "saved_scale", _torch.float32,
                    (R, 2 * _scale_shape(R, W, True)[1]), dev)
    _call(_fx.lib().mslkb_swiglu_quant_backward(
        _dense(dy, "dy", dy.dtype, (R, W), dev), kp, sp,
        _dense(out, "out", dy.dtype, (R, 2 * W), dev), R, W, dt, s.raw),
        "swiglu_quant_backward")
    return out
