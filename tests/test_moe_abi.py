"""C entry points of the operators around the grouped product, without a GPU: argument errors
come before any CUDA call, empty calls do nothing, workspace sizes."""
import pytest

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from fp8_rowwise_scaled_gb300 import moe

P = 256  # a pointer that no call here follows


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fxbuild.build()
    fx.lib()


def call(fn, defaults):
    def run(**kw):
        assert not set(kw) - set(defaults), kw
        return fn(*[kw.get(k, d) for k, d in defaults.items()])
    return run


norm = call(fx.mslkb_add_rms_norm_quant, dict(
    x=P, residual=P, weight=P, q=P, scale=P, residual_out=P, y=P, rstd=P, T=2, H=256, ldx=256,
    ldr=256, eps=1e-6, dtype=moe.MSLKB_BF16, weight_fp32=0, groupwise=0, stream=0))
norm_backward = call(fx.mslkb_add_rms_norm_quant_backward, dict(
    dy=P, h=P, weight=P, rstd=P, dresidual=P, dx=P, dweight=P, workspace=P, bytes=1 << 20, T=2,
    H=256, dtype=moe.MSLKB_BF16, weight_fp32=0, stream=0))
route = call(fx.mslkb_route_experts, dict(
    logits=P, bias=P, ids=P, weights=P, T=2, E=16, ld=16, top_k=2, score=moe.MSLKB_SIGMOID,
    groups=4, top_groups=2, group_top=2, renormalize=1, scale=1.0, dtype=moe.MSLKB_FP32, stream=0))
route_backward = call(fx.mslkb_route_experts_backward, dict(
    dweights=P, logits=P, ids=P, dlogits=P, T=2, E=16, ld=16, top_k=2, score=moe.MSLKB_SOFTMAX,
    renormalize=1, scale=1.0, dtype=moe.MSLKB_FP32, stream=0))
dispatch = call(fx.mslkb_moe_dispatch, dict(
    x=P, x_scale=P, ids=P, x_out=P, scale_out=P, m_sizes=P, dest=P, T=4, top_k=2, E=16, row_bytes=256, scale_cols=1, stream=0))
combine = call(fx.mslkb_moe_combine, dict(
    rows=P, dest=P, weights=P, out=P, T=4, top_k=2, H=256, R=8, dtype=moe.MSLKB_BF16, stream=0))
combine_backward = call(fx.mslkb_moe_combine_backward, dict(
    dout=P, rows=P, dest=P, weights=P, drows=P, dweights=P, T=4, top_k=2, H=256, R=8,
    dtype=moe.MSLKB_BF16, stream=0))
swiglu = call(fx.mslkb_swiglu_quant, dict(
    x=P, q=P, scale=P, saved=P, saved_scale=P, R=2, W=256, ldx=512, dtype=moe.MSLKB_BF16,
    groupwise=0, stream=0))
swiglu_backward = call(fx.mslkb_swiglu_quant_backward, dict(
    dy=P, saved=P, saved_scale=P, dx=P, R=2, W=256, dtype=moe.MSLKB_BF16, stream=0))


def refused(fn, status, *cases):
    for kw in cases:
        assert fn(**kw) == status, (kw, fx.mslkb_status_string(status))


def test_null_pointers():
    refused(norm, fx.MSLKB_ERR_NULL, *({k: None} for k in ("x", "weight", "q", "scale")))
    refused(norm_backward, fx.MSLKB_ERR_NULL,
            *({k: None} for k in ("dy", "h", "weight", "rstd", "dx", "dweight")))
    refused(route, fx.MSLKB_ERR_NULL, *({k: None} for k in ("logits", "ids", "weights")))
    refused(route_backward, fx.MSLKB_ERR_NULL,
            *({k: None} for k in ("dweights", "logits", "ids", "dlogits")))
    refused(dispatch, fx.MSLKB_ERR_NULL,
            *({k: None} for k in ("x", "x_scale", "ids", "x_out", "scale_out", "m_sizes", "dest")))
    refused(combine, fx.MSLKB_ERR_NULL, *({k: None} for k in ("rows", "dest", "out")))
    refused(combine_backward, fx.MSLKB_ERR_NULL,
            *({k: None} for k in ("dout", "rows", "dest", "weights", "drows", "dweights")))
    refused(swiglu, fx.MSLKB_ERR_NULL, *({k: None} for k in ("x", "q", "scale", "saved_scale")))
    refused(swiglu_backward, fx.MSLKB_ERR_NULL, *({k: None} for k in ("dy", "saved", "dx")))


def test_sizes():
    big = 1 << 33
    refused(norm, fx.MSLKB_ERR_SHAPE, dict(T=-1), dict(H=-1), dict(T=big), dict(H=32769, ldx=32769),
            dict(ldx=255), dict(ldr=255), dict(H=200, groupwise=1), dict(eps=0.0), dict(eps=1.0),
            dict(eps=float("nan")), dict(eps=-1e-6))
    refused(norm_backward, fx.MSLKB_ERR_SHAPE, dict(T=-1), dict(H=-1), dict(H=32769))
    refused(route, fx.MSLKB_ERR_SHAPE, dict(T=-1), dict(E=1025, ld=1025), dict(top_k=17),
            dict(E=64, ld=64, top_k=33, groups=1, top_groups=1), dict(ld=15), dict(groups=0),
            dict(groups=3), dict(groups=33), dict(top_groups=0), dict(top_groups=5), dict(top_k=9),
            dict(group_top=0), dict(group_top=3), dict(score=2), dict(scale=float("nan")))
    refused(route_backward, fx.MSLKB_ERR_SHAPE, dict(T=-1), dict(top_k=17), dict(ld=15),
            dict(score=-1))
    refused(dispatch, fx.MSLKB_ERR_SHAPE, dict(T=-1), dict(top_k=33), dict(E=1025),
            dict(row_bytes=-1), dict(row_bytes=big), dict(scale_cols=-1), dict(T=1 << 30, top_k=4))
    refused(combine, fx.MSLKB_ERR_SHAPE, dict(T=-1), dict(top_k=33), dict(H=-1), dict(R=-1),
            dict(H=big), dict(R=big))
    refused(combine_backward, fx.MSLKB_ERR_SHAPE, dict(T=-1), dict(top_k=33), dict(H=-1))
    refused(swiglu, fx.MSLKB_ERR_SHAPE, dict(R=-1), dict(W=32896, ldx=2 * 32896), dict(ldx=511),
            dict(W=200), dict(W=200, saved=None, groupwise=1))
    refused(swiglu_backward, fx.MSLKB_ERR_SHAPE, dict(R=-1), dict(W=200))


def test_types_and_workspaces():
    for fn in (norm, norm_backward, route, route_backward, combine, combine_backward, swiglu,
               swiglu_backward):
        refused(fn, fx.MSLKB_ERR_DTYPE, dict(dtype=3), dict(dtype=-1))
    need = fx.mslkb_add_rms_norm_quant_backward_workspace_bytes(2, 256)
    assert need >= 2 * 256 * 4
    refused(norm_backward, fx.MSLKB_ERR_WORKSPACE, dict(workspace=None), dict(workspace=264),
            dict(bytes=need - 1))
    assert fx.mslkb_add_rms_norm_quant_backward_workspace_bytes(0, 256) == 0
    assert fx.mslkb_add_rms_norm_quant_backward_workspace_bytes(1 << 20, 32768) <= 608 * 32768 * 4


def test_nothing_to_do():
    none = dict.fromkeys
    assert norm(T=0, **none(("x", "weight", "q", "scale"))) == fx.MSLKB_OK
    assert norm(H=0, ldx=0, ldr=0) == fx.MSLKB_OK
    assert norm_backward(H=0, dweight=None) == fx.MSLKB_OK
    assert route(T=0, logits=None) == fx.MSLKB_OK and route(top_k=0, ids=None) == fx.MSLKB_OK
    assert route_backward(T=0, logits=None) == fx.MSLKB_OK
    assert combine(T=0, out=None) == fx.MSLKB_OK and combine(H=0, out=None) == fx.MSLKB_OK
    assert combine_backward(T=0, dout=None) == fx.MSLKB_OK
    assert swiglu(R=0, x=None) == fx.MSLKB_OK and swiglu(W=0, ldx=0) == fx.MSLKB_OK
    assert swiglu_backward(R=0, dy=None) == fx.MSLKB_OK


def test_new_status_strings():
    for s in (fx.MSLKB_ERR_DTYPE, fx.MSLKB_ERR_WORKSPACE):
        assert fx.mslkb_status_string(s) not in ("unknown status", "ok")


def test_rows_too_long_and_rows_written_over():
    refused(dispatch, fx.MSLKB_ERR_SHAPE, dict(row_bytes=(1 << 30) + 1),
            dict(scale_cols=(1 << 30) + 1))
    # in place, the rows of the sum have to lie where the residual's were
    refused(norm, fx.MSLKB_ERR_SHAPE, dict(ldr=257))
