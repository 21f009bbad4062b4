"""More of the operators around the grouped product on the GPU: what tests/test_moe_ops.py does
not reach, with its helpers and the same 64-bit forms."""
import threading

import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
import moe_reference as ref
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import U, close, np64, rounding
from route_tolerance import route_backward_tolerance
from test_moe_ops import (BF16, EPS, FP16, FP32, flat, gen, moe_step, randn, shifted,
                          strided)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


@pytest.mark.parametrize("T,H", [(2900, 136), (3000, 264), (2000, 520), (1900, 1000), (1700, 1032),
                                 (1500, 2056), (900, 4104), (700, 5128), (800, 8192)])
@pytest.mark.parametrize("with_res", [True, False])
def test_norm_backward_fp32_many_rows_per_cta(T, H, with_res):
    """32-bit rows through the ring, several per CTA, most with a last warp partly past the row's
    end: right, and the same bits every time."""
    g = gen(T + H)
    dy, h, w = randn(g, T, H), randn(g, T, H, scale=2.0), randn(g, H)
    dres = randn(g, T, H) if with_res else None
    rstd = h.double().square().mean(-1).add(EPS).rsqrt().float()
    dx, dw = fx.add_rms_norm_quant_backward(dy, h, w, rstd, dres)
    a = [np64(t) for t in (dy, h, w, rstd)]
    want_dx, want_dw = ref.norm_backward(*a, None if dres is None else np64(dres))
    xhat, gg = a[1] * a[3][:, None], a[0] * a[2]
    size = a[3][:, None] * (np.abs(gg) + np.abs(xhat) * np.abs(gg * xhat).mean(-1, keepdims=True))
    close(dx, want_dx, 48 * U * size + 2 * U * np.abs(want_dx), "dx")
    # additions: a thread's rows, up to 16 rows side by side, up to 19 partial sums a warp, 32
    # warps; and the roundings of h * rstd and of the product
    close(dw, want_dw, (T // 152 + 1 + 16 + 19 + 32 + 2) * U * np.abs(a[0] * xhat).sum(0), "dweight")
    for _ in range(20):
        again = fx.add_rms_norm_quant_backward(dy, h, w, rstd, dres)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw), "not the same bits again"


# ---------------------------------------------------------------------------------------
# SwiGLU's gradient in 32 bits
# ---------------------------------------------------------------------------------------
def check_swiglu_backward_fp32(dx, dy, values):
    """Each element of an fp32 gradient to the roundings of its own formula, u = 2^-24 each: the
    exponential 2, 1 + e and its inverse 1 each, so that sigmoid(gate) and sigmoid(-gate) are good
    to 6 (3 and 2 with one product more); dup two products beside (8), dgate three and the sum
    1 + gate sigmoid(-gate).  One more for the terms of second order; and the spacing of the
    subnormals, 2^-149, in the exponential and the products."""
    gate, up = np.split(values, 2, axis=1)
    s, rest = ref.sigmoid(gate), ref.sigmoid(-gate)
    factor = 1 + gate * rest
    want = np.concatenate([dy * up * s * factor, dy * gate * s], axis=1)
    tol = np.concatenate([np.abs(dy * up) * s * (11 * np.abs(factor) + 7 * np.abs(gate) * rest) * U,
                          9 * U * np.abs(dy * gate) * s], axis=1)
    small = (1 + np.abs(dy)) * (1 + np.abs(gate)) * (1 + np.abs(up)) * 2.0 ** -147
    close(dx, want, tol + np.concatenate([small, small], axis=1), "dx")


@pytest.mark.parametrize("R,W", [(40, 256), (7, 1000), (5, 125), (3, 8192)])
@pytest.mark.parametrize("reach", [3.0, 20.0, 86.0, 110.0])
def test_swiglu_backward_fp32_is_full_precision(R, W, reach):
    """Gates over [-reach, reach], from the input and, in whole blocks, from its checkpoint."""
    g = gen(R + W)
    x, dy = randn(g, R, 2 * W), randn(g, R, W)
    x[:, :W] = (2 * torch.rand((R, W), generator=g, device="cuda") - 1) * reach
    check_swiglu_backward_fp32(fx.swiglu_quant_backward(dy, x), np64(dy), np64(x))
    check_swiglu_backward_fp32(fx.swiglu_quant_backward(shifted(dy), x), np64(dy), np64(x))
    if W % ref.BLOCK == 0:
        kept = fx.swiglu_quant(x, checkpoint=True)
        values = np64(kept.saved).reshape(R, -1, ref.BLOCK) * np64(kept.saved_scale)[..., None]
        # (the kernel's product of code and scale is rounded to fp32)
        values = values.reshape(R, 2 * W).astype(np.float32).astype(np.float64)
        check_swiglu_backward_fp32(fx.swiglu_quant_backward(dy, kept.saved, kept.saved_scale),
                                   np64(dy), values)


def test_swiglu_backward_fp32_extremes():
    """Infinite and NaN gates as in the formula, and gates where sigmoid is a subnormal."""
    gate = [-104.0, -103.0, -95.0, -88.5, -87.5, 0.0, -0.0, 88.5, 104.0, 200.0, -200.0]
    x = torch.tensor([gate + [1.0] * len(gate)], device="cuda")
    dy = torch.ones((1, len(gate)), device="cuda")
    check_swiglu_backward_fp32(fx.swiglu_quant_backward(dy, x), np64(dy), np64(x))
    x[0, 0], x[0, 1] = float("nan"), float("inf")
    dx = fx.swiglu_quant_backward(dy, x)[0]
    n = len(gate)
    assert torch.isnan(dx[0]) and torch.isnan(dx[n]) and torch.isinf(dx[n + 1])
    assert torch.isfinite(dx[2:n]).all() and torch.isfinite(dx[n + 2:]).all()


# ---------------------------------------------------------------------------------------
# routing gradient, element by element
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False),
                                          ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("T,E,k", [(33, 8, 2), (9, 31, 6), (21, 33, 4), (21, 64, 6), (13, 100, 7),
                                   (37, 128, 8), (21, 160, 6), (21, 161, 6), (30, 256, 8),
                                   (11, 300, 10), (21, 384, 8), (9, 500, 10), (9, 512, 20),
                                   (5, 777, 8), (5, 1024, 32)])
def test_route_backward_element_by_element(T, E, k, score, renorm, dtype):
    """Every number of experts per lane, whole and broken pieces; logits as slices of wider rows,
    off their alignment, and the gradient off its own (which deals the experts to the lanes in
    another order: the same bound, not the same bits)."""
    g = gen(T + E)
    x = randn(g, T, E, dtype=dtype, scale=1.5)
    ids = fx.route_experts(x, k, score=score, renormalize=renorm).ids
    ids[T // 2, 0] = -1
    ids[0, -1] = E + 3
    x[1, torch.randperm(E, generator=g, device="cuda")[:E // 4]] = float("-inf")
    dw = randn(g, T, k)
    kw = dict(score=score, renormalize=renorm, scale=1.25)
    dx = fx.route_experts_backward(dw, x, ids, **kw)
    args = np64(dw), np64(x), np64(ids), score == "sigmoid", renorm, 1.25
    want = ref.route_backward(*args)
    tol = route_backward_tolerance(*args, dtype, want)
    close(dx, want, tol, "dlogits")
    for v in (strided(x, 8), strided(x, 3), shifted(x)):
        close(fx.route_experts_backward(dw, v, ids, **kw), want, tol, "dlogits of other rows")
    out = shifted(torch.zeros_like(dx))
    assert fx.route_experts_backward(dw, x, ids, out=out, **kw) is out
    close(out, want, tol, "dlogits off their alignment")


def test_calls_of_several_threads():
    """Host threads on streams and data of their own at the same time."""
    g = gen(91)
    E, n, cases = 32, 4, []
    for T in (3, 65, 400, 700):
        cases.append((randn(g, T, 512, dtype=BF16), randn(g, T, 512, dtype=BF16),
                      randn(g, 512, dtype=BF16), randn(g, T, E)))
    want = [flat(moe_step(*c, E)) for c in cases]
    grads = [fx.add_rms_norm_quant_backward(c[0], c[1], c[2], torch.ones(len(c[0]), device="cuda"))
             for c in cases]
    torch.cuda.synchronize()
    wrong, gate = [], threading.Barrier(n)

    def body(i):
        gate.wait()
        try:
            stream = torch.cuda.Stream()
            ones = torch.ones(len(cases[i][0]), device="cuda")
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                for _ in range(30):
                    got = flat(moe_step(*cases[i], E))
                    grad = fx.add_rms_norm_quant_backward(*cases[i][:3], ones)
                    same = [torch.equal(a, b) for a, b in zip(got + list(grad), want[i] + list(grads[i]))]
                    if not all(same):
                        wrong.append((i, same))
            stream.synchronize()
        except BaseException as e:
            wrong.append((i, e))
    threads = [threading.Thread(target=body, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
    assert fx.device_status() == 0


@pytest.mark.parametrize("groupwise", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_rows_without_columns(groupwise, given):
    """Rows of no columns have no codes, and their scales are those of zeros, 1, not what the
    memory held; rstd is that of a sum of squares of zero."""
    T = 300
    x, w = torch.zeros((T, 0), dtype=BF16, device="cuda"), torch.ones(0, dtype=BF16, device="cuda")
    scales = (T, 0) if groupwise else (T,)

    def poison():
        held = [torch.full(scales if i else (T,), float("nan"), device="cuda") for i in range(2)]
        return (held[1], held[0]) if given else (None, None)   # else back to the allocator
    q = torch.zeros((T, 0), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        scale, rstd = poison()
        out = fx.NormQuant(q, scale, None, None, rstd) if given else None
        torch.cuda.synchronize()
        got = fx.add_rms_norm_quant(x, w, groupwise=groupwise, want_rstd=True, out=out, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got.scale, torch.ones(scales, device="cuda"))
        close(got.rstd, np.full(T, EPS ** -0.5), 4 * U * EPS ** -0.5, "rstd")
        scale, _ = poison()
        out = fx.SwigluQuant(q, scale, None, None) if given else None
        torch.cuda.synchronize()
        got = fx.swiglu_quant(x, groupwise=groupwise, out=out, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got.scale, torch.ones(scales, device="cuda"))


def test_sizes_are_refused_before_results_are_allocated():
    """Numbers of experts out of range, as ValueError and with no memory taken first (the results
    that they name would have been up to a terabyte)."""
    x = torch.zeros((4096, 64), device="cuda")
    ids = torch.zeros((4096, 2), dtype=torch.int32, device="cuda")
    wide = torch.zeros((4096, 1000), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for call in (lambda: fx.route_experts(x, -1), lambda: fx.route_experts(x, 33),
                 lambda: fx.route_experts(x, 10 ** 8), lambda: fx.moe_dispatch(x, None, ids, -1),
                 lambda: fx.moe_dispatch(x, None, ids, 10 ** 11),
                 lambda: fx.moe_dispatch(x, None, wide, 8)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fx.moe_dispatch(x, [1.0], ids, 8)
    assert torch.cuda.max_memory_allocated() == before


def test_no_memory_for_the_norm_gradient():
    """The scratch of a call raises as torch's own allocations do, and the next call is fine."""
    T, H = 700, 16384    # 608 rows of partial sums: 40 MB
    x, w = torch.zeros((T, H), dtype=BF16, device="cuda"), torch.ones(H, dtype=BF16, device="cuda")
    rstd = torch.ones(T, device="cuda")
    out = (torch.empty_like(x), torch.empty(H, device="cuda"))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    try:
        torch.cuda.set_per_process_memory_fraction(0.0)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            torch.empty(40 << 20, device="cuda")
        with pytest.raises(torch.cuda.OutOfMemoryError):
            fx.add_rms_norm_quant_backward(x, x, w, rstd, out=out)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    dx, dw = fx.add_rms_norm_quant_backward(x, x, w, rstd, out=out)
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_nan_bias(score):
    """An expert with a NaN bias is taken first, with the weight that its logit gives."""
    g = gen(92)
    x, bias = randn(g, 20, 64), torch.zeros(64, device="cuda")
    bias[11] = float("nan")
    out = fx.route_experts(x, 4, bias=bias, score=score)
    assert (out.ids[:, 0] == 11).all() and torch.isfinite(out.weights).all()
    want = ref.route_weights(np64(x), np64(out.ids), score == "sigmoid", True, 1.0)
    close(out.weights, want, 64 * U * want, "weights")   # as in tests/test_moe_ops.py
