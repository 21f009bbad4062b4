"""The operators around the grouped product on the GPU, against plain 64-bit forms
(moe_reference): norm with e4m3 output, expert routing, dispatch and combine, SwiGLU with an
e4m3 output and checkpoint, and their gradients (against the formulas and against
differences); ragged and odd sizes, strides, alignments, masks that leave nothing, streams,
graphs, refusals."""
import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
import moe_reference as ref
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import U, close, np64, rounding

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6
REL = 32 * U      # the norm's relative error: half of the 42 u of its sum, and 8 roundings


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=FP32, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def shifted(t):
    """The same values one element into a buffer: aligned for the element type only."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = b[1:].view(t.shape)
    v.copy_(t)
    return v


def strided(t, extra):
    """The same rows as slices of rows that are `extra` elements longer."""
    b = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


# ---------------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------------
def check_norm(out, x, residual, weight, groupwise, eps=EPS, want_y=True, want_rstd=True):
    h, rstd, y = ref.norm(np64(x), None if residual is None else np64(residual), np64(weight), eps)
    ref.check_codes(out.q, out.scale, y, ref.BLOCK if groupwise else x.shape[1], REL, "q")
    if residual is None:
        assert out.residual is None
    else:
        close(out.residual, h, rounding(x.dtype, h) + 2 * U * np.abs(h), "residual")
    if want_y:
        close(out.y, y, rounding(x.dtype, y) + REL * np.abs(y), "y")
    if want_rstd:
        close(out.rstd, rstd, REL * rstd, "rstd")


NORM_CASES = [  # tokens, hidden, groupwise
    (1, 1, False), (3, 7, False), (5, 128, True), (1, 7168, False), (2, 7168, True),
    (7, 1000, False), (4, 1025, False), (17, 8192, True), (3, 8200, False), (2, 16384, True),
    (2, 16392, False), (2, 32768, True), (1, 32768, False), (2, 32767, False), (300, 256, True),
    # many rows: the persistent kernel, CTAs with several rows and with one
    (609, 7168, False), (1500, 8192, True), (2000, 128, True), (1300, 1000, False),
    (700, 4096, False), (1250, 4104, False), (620, 16384, True), (640, 12304, False),
    (650, 1025, False), (300, 8, False), (700, 33, False)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H,groupwise", NORM_CASES)
def test_norm(T, H, groupwise, dtype):
    g = gen(T * 1000 + H)
    x, res = randn(g, T, H, dtype=dtype, scale=2.0), randn(g, T, H, dtype=dtype)
    w = randn(g, H).mul_(0.3).add_(1).to(dtype)
    out = fx.add_rms_norm_quant(x, w, res, eps=EPS, groupwise=groupwise, want_y=True, want_rstd=True)
    check_norm(out, x, res, w, groupwise)


@pytest.mark.parametrize("T,H,groupwise", [(1, 7168, False), (6, 384, True), (3, 77, False)])
def test_norm_plain_inputs(T, H, groupwise):
    """No residual, nothing beside the codes; fp32 weight beside bf16 rows; other eps."""
    g = gen(5)
    x, w = randn(g, T, H, dtype=BF16), randn(g, H)
    out = fx.add_rms_norm_quant(x, w, eps=1e-3, groupwise=groupwise)
    assert out.y is None and out.rstd is None and out.residual is None
    check_norm(out, x, None, w, groupwise, eps=1e-3, want_y=False, want_rstd=False)


@pytest.mark.parametrize("H,groupwise", [(512, True), (1000, False), (7168, False)])
def test_norm_strides_and_alignment(H, groupwise):
    g = gen(6)
    T = 9
    x, res = randn(g, T, H, dtype=BF16), randn(g, T, H, dtype=BF16)
    w = randn(g, H, dtype=BF16)
    want = fx.add_rms_norm_quant(x, w, res, groupwise=groupwise, want_y=True, want_rstd=True)
    check_norm(want, x, res, w, groupwise)
    for xs, rs, ws in ((strided(x, 8), strided(res, 24), w), (strided(x, 1), res, w),
                       (shifted(x), res, w), (x, shifted(res), shifted(w))):
        got = fx.add_rms_norm_quant(xs, ws, rs, groupwise=groupwise, want_y=True, want_rstd=True)
        check_norm(got, x, res, w, groupwise)
    # outputs that only suit their element type
    out = fx.NormQuant(shifted(want.q.view(torch.uint8)), want.scale, shifted(want.residual),
                       shifted(want.y), want.rstd)
    for t in (out.q, out.residual, out.y):
        t.zero_()
    got = fx.add_rms_norm_quant(x, w, res, groupwise=groupwise, want_y=True, want_rstd=True, out=out)
    assert got is out
    check_norm(out, x, res, w, groupwise)


def test_norm_residual_in_place():
    g = gen(7)
    T, H = 33, 7168
    x, res = randn(g, T, H, dtype=BF16), randn(g, T, H, dtype=BF16)
    w = randn(g, H, dtype=BF16)
    want = fx.add_rms_norm_quant(x, w, res)
    stream = res.clone()
    out = fx.NormQuant(torch.empty_like(want.q), torch.empty_like(want.scale), stream, None, None)
    fx.add_rms_norm_quant(x, w, stream, out=out)
    assert torch.equal(stream, want.residual)
    assert torch.equal(out.q.view(torch.uint8), want.q.view(torch.uint8))
    assert torch.equal(out.scale, want.scale)


def test_norm_extremes():
    """Rows of zeros, of the smallest and of large values, a weight of zeros, NaN and infinity:
    each stays in its row (its block, for a NaN weight)."""
    H = 256
    x = torch.zeros(8, H, dtype=FP32, device="cuda")
    g = gen(8)
    x[1] = randn(g, H)
    x[2] = 1e-38
    x[3] = randn(g, H) * 1e15
    x[4] = randn(g, H)
    x[4, 3] = float("nan")
    x[5] = randn(g, H)
    x[5, 200] = float("inf")
    x[6, 255] = -3.0
    x[7] = randn(g, H) * 1e-30
    w = randn(g, H)
    for groupwise in (False, True):
        out = fx.add_rms_norm_quant(x, w, groupwise=groupwise, want_y=True, want_rstd=True)
        fine = torch.tensor([0, 1, 2, 3, 6, 7], device="cuda")
        check_norm(fx.NormQuant(out.q[fine], out.scale[fine], None, out.y[fine], out.rstd[fine]),
                   x[fine], None, w, groupwise)
        scale = out.scale.reshape(8, -1)
        assert torch.isnan(scale[4]).all() and torch.isnan(out.y[4]).all()
        assert torch.isnan(scale[5, -1]) and torch.isnan(out.y[5, 200])
        assert torch.equal(out.q[0].float(), torch.zeros(H, device="cuda"))
        assert torch.equal(scale[0], torch.ones_like(scale[0]))
    zero = fx.add_rms_norm_quant(x[1:2], torch.zeros_like(w))
    assert zero.scale.item() == 1 and not zero.q.float().any()
    w[130] = float("nan")
    out = fx.add_rms_norm_quant(x[1:2], w, groupwise=True)
    assert torch.isfinite(out.scale[0, 0]) and torch.isnan(out.scale[0, 1])


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H,with_res", [(1, 1, True), (3, 129, False), (1, 7168, True),
                                          (700, 512, True), (50, 1000, False), (5, 16384, True),
                                          (4, 32768, True), (3, 32767, False),
                                          (1216, 7168, True), (900, 8192, False),
                                          (1000, 136, True), (305, 4096, True),
                                          (1300, 1025, True), (2500, 128, True),
                                          (1501, 2048, False), (700, 16384, True),
                                          (310, 8, False), (999, 1000, True)])
def test_norm_backward(T, H, with_res, dtype):
    g = gen(T + H)
    dy, h = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype, scale=2.0)
    w = randn(g, H, dtype=dtype)
    dres = randn(g, T, H, dtype=dtype) if with_res else None
    rstd = h.double().square().mean(-1).add(EPS).rsqrt().float()
    dx, dw = fx.add_rms_norm_quant_backward(dy, h, w, rstd, dres)
    a = [np64(t) for t in (dy, h, w, rstd)]
    want_dx, want_dw = ref.norm_backward(*a, None if dres is None else np64(dres))
    xhat, gg = a[1] * a[3][:, None], a[0] * a[2]
    size = a[3][:, None] * (np.abs(gg) + np.abs(xhat) * np.abs(gg * xhat).mean(-1, keepdims=True))
    # 42 u of the mean's terms, and the roundings of the other terms
    close(dx, want_dx, rounding(dtype, want_dx) + 48 * U * size + 2 * U * np.abs(want_dx), "dx")
    # a CTA's rows (two at most here), 608 / 8 rows of partial sums and 8 groups: 86 additions
    close(dw, want_dw, 96 * U * np.abs(a[0] * xhat).sum(0), "dweight")
    again = fx.add_rms_norm_quant_backward(dy, h, w, rstd, dres)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw), "not the same bits again"
    # in place of the incoming gradients
    out = (dy.clone(), torch.empty_like(dw))
    fx.add_rms_norm_quant_backward(out[0], h, w, rstd, dres, out=out)
    assert torch.equal(out[0], dx) and torch.equal(out[1], dw)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,H,with_res", [(1000, 256, True), (1001, 264, False), (700, 520, True),
                                          (2600, 768, True), (170, 1024, True), (160, 2048, True),
                                          (1300, 1536, False), (400, 2056, True),
                                          (333, 5120, True), (333, 5128, False), (320, 6144, True),
                                          (310, 8192, True), (153, 8192, False), (2000, 129, True),
                                          (700, 513, False), (300, 769, True), (151, 33, True),
                                          (32, 4096, True), (41, 7168, False), (90, 8192, True),
                                          (161, 2064, True), (31, 5120, True), (2, 24, True)])
def test_norm_backward_of_many_widths(T, H, with_res, dtype):
    test_norm_backward(T, H, with_res, dtype)


def test_norm_backward_unaligned_and_fp32_weight():
    g = gen(3)
    T, H = 11, 512
    dy, h, dres = (randn(g, T, H, dtype=BF16) for _ in range(3))
    w = randn(g, H)
    rstd = h.double().square().mean(-1).add(EPS).rsqrt().float()
    dx, dw = fx.add_rms_norm_quant_backward(dy, h, w, rstd, dres)
    dx2, dw2 = fx.add_rms_norm_quant_backward(shifted(dy), h, shifted(w), rstd, shifted(dres))
    close(dx2, np64(dx), 2.0 ** -7 * np.abs(np64(dx)) + 1e-6, "dx")
    close(dw2, np64(dw), 1e-5 * np.abs(np64(dw)) + 1e-5, "dweight")


def test_norm_backward_against_differences():
    """The gradient of sum(y * dy) + sum(h * dres) by central differences of the 64-bit form."""
    g = gen(4)
    T, H = 3, 24
    x, res, dy, dres = (randn(g, T, H) for _ in range(4))
    w = randn(g, H)
    out = fx.add_rms_norm_quant(x, w, res, want_y=True, want_rstd=True)
    dx, dw = fx.add_rms_norm_quant_backward(dy, out.residual, w, out.rstd, dres)

    def loss(xv, wv):
        h, _, y = ref.norm(xv, np64(res), wv, EPS)
        return (y * np64(dy)).sum() + (h * np64(dres)).sum()

    check_differences(lambda v: loss(v, np64(w)), np64(x), np64(dx))
    check_differences(lambda v: loss(np64(x), v), np64(w), np64(dw))


def check_differences(f, at, grad, step=1e-5):
    """Central differences: error step^2 * (third derivative) / 6 and 2^-52 * |f| / step,
    beside the kernel's own fp32 error: 1e-5 of the gradient's size in all."""
    flat = at.reshape(-1)
    size = np.abs(grad).max() + 1e-3
    for i in range(flat.size):
        up, down = flat.copy(), flat.copy()
        up[i] += step
        down[i] -= step
        d = (f(up.reshape(at.shape)) - f(down.reshape(at.shape))) / (2 * step)
        assert abs(d - grad.reshape(-1)[i]) <= 1e-5 * size, (i, d, grad.reshape(-1)[i])


# ---------------------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------------------
WEIGHT_TOL = 64 * U   # exp and the score's roundings: (|x - max| <= 20) + 2 ulp of exp + sums

ROUTE_CASES = [  # E, k, groups, top_groups, group_top
    (256, 8, 8, 4, 2), (256, 8, 1, 1, 1), (160, 6, 8, 3, 1), (64, 2, 1, 1, 1), (8, 2, 4, 2, 2),
    (31, 5, 1, 1, 1), (500, 10, 4, 2, 2), (384, 8, 1, 1, 1), (1024, 32, 32, 8, 2), (1, 1, 1, 1, 1),
    (33, 4, 3, 2, 1), (96, 8, 6, 2, 2), (40, 40 // 5, 5, 1, 1), (128, 1, 2, 1, 1), (6, 6, 1, 1, 1)]


def tied_logits(g, T, E):
    """Logits of few distinct values: ties of experts everywhere, near-ties of experts nowhere
    (sums of two may tie by the sigmoid's symmetry: see tied_groups)."""
    return torch.randint(-4, 5, (T, E), generator=g, device="cuda").float() * 0.5


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("E,k,groups,top_groups,group_top", ROUTE_CASES)
def test_route(E, k, groups, top_groups, group_top, dtype, score):
    g = gen(E + k)
    for T, renorm, with_bias in ((1, True, False), (37, False, True), (130, True, True)):
        x = tied_logits(g, T, E).to(dtype)
        bias = torch.randint(-3, 4, (E,), generator=g, device="cuda").float() / 8 \
            if with_bias else None
        out = fx.route_experts(x, k, bias=bias, score=score, num_groups=groups,
                               topk_groups=top_groups, group_top=group_top, renormalize=renorm,
                               scale=2.5)
        ids, weights = ref.route(np64(x), None if bias is None else np64(bias), k,
                                 score == "sigmoid", groups, top_groups, group_top, renorm, 2.5)
        choice, worth = choices(x, bias, score, groups, group_top)
        either = tied_groups(worth, top_groups)      # decided by the last bit: either way is right
        if score == "softmax" and with_bias:
            either[:] = True
        check_choice(np64(out.ids)[either], choice[either], worth[either], top_groups)
        ids[either] = np64(out.ids)[either]
        weights[either] = ref.route_weights(np64(x), ids, score == "sigmoid", renorm, 2.5)[either]
        assert np.array_equal(np64(out.ids), ids), f"T={T} renorm={renorm}"
        close(out.weights, weights, WEIGHT_TOL * weights, "weights")


def choices(x, bias, score, groups, group_top):
    """The 64-bit choice values [T, E] and what the groups are worth [T, groups]."""
    x = np64(x)
    if score == "sigmoid":
        choice = ref.sigmoid(x)
    else:
        e = np.exp(x - x.max(-1, keepdims=True))
        choice = e / e.sum(-1, keepdims=True)
    if bias is not None:
        choice = choice + np64(bias)
    per = np.sort(choice.reshape(x.shape[0], groups, -1), -1)[..., ::-1]
    return choice, per[..., :group_top].sum(-1)


def tied_groups(worth, top_groups):
    """Rows where the last group in and the first one out agree to 1e-6 but not exactly the
    same way in 32 and 64 bits (sigmoid(a) + sigmoid(-a) = 1 for every a)."""
    w = np.sort(worth, -1)[:, ::-1]
    if top_groups == w.shape[1]:
        return np.zeros(w.shape[0], bool)
    return np.abs(w[:, top_groups - 1] - w[:, top_groups]) < 1e-6


def check_choice(ids, choice, worth, top_groups):
    """A choice in which values that agree to fp32 may be taken either way: the chosen values
    do not rise, the groups are the best, nothing left out is above the last one."""
    E, groups = choice.shape[1], worth.shape[1]
    for t in range(len(ids)):
        assert len(set(ids[t])) == ids.shape[1] and (ids[t] >= 0).all()
        mine = choice[t, ids[t]]
        assert (np.diff(mine) <= 1e-6).all()
        used = sorted(set(ids[t] // (E // groups)))
        assert len(used) <= top_groups
        cut = np.sort(worth[t])[::-1][top_groups - 1]
        assert (worth[t, used] >= cut - 1e-6).all()
        surely = worth[t] > cut + 1e-6    # groups that are in without doubt
        rest = [i for i in range(E) if i not in set(ids[t]) and surely[i // (E // groups)]]
        assert not rest or choice[t, rest].max() <= mine.min() + 1e-6


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_random_logits(score, renorm):
    """Continuous logits (no ties): the choice of the 64-bit scores, whose gaps are checked to
    be wider than fp32's error."""
    g = gen(77)
    x = 2 * torch.randn((257, 200), generator=g, device="cuda")
    out = fx.route_experts(x, 8, score=score, renormalize=renorm)
    ids, weights = ref.route(np64(x), None, 8, score == "sigmoid", 1, 1, 1, renorm, 1.0)
    s = np.sort(ref.sigmoid(np64(x)) if score == "sigmoid" else np64(x), -1)[:, ::-1]
    clear = (s[:, :8] - s[:, 1:9]).min(-1) > 4e-7
    assert clear.sum() > 200
    assert np.array_equal(np64(out.ids)[clear], ids[clear])
    close(out.weights[torch.from_numpy(clear).cuda()], weights[clear],
          WEIGHT_TOL * weights[clear], "weights")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 4, 5])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masks(score, groups, renorm):
    """Experts masked by -inf: rows with fewer than top_k left, rows with none, groups with one
    left or none; a bias of -inf masks as well; the type's lowest value is a number."""
    g = gen(9)
    T, E, k = 60, 40, 6
    x = tied_logits(g, T, E)
    x[torch.rand((T, E), generator=g, device="cuda") < 0.6] = float("-inf")
    x[3] = float("-inf")
    x[4] = float("-inf")
    x[4, 39] = 1.0
    x[5, :] = torch.finfo(FP32).min
    x[6, :30] = torch.finfo(FP32).min
    if score == "softmax":
        x[7, 1] = -300.0          # underflows beside 0, and is still a choice
        x[7, 2] = -200.0
    kw = dict(num_groups=groups, topk_groups=min(groups, 2))
    out = fx.route_experts(x, k, score=score, renormalize=renorm, **kw)
    ids, weights = ref.route(np64(x), None, k, score == "sigmoid", groups, min(groups, 2), 1,
                             renorm, 1.0)
    assert np.array_equal(np64(out.ids), ids)
    close(out.weights, weights, WEIGHT_TOL * weights + 2.0 ** -126, "weights")
    assert (np64(out.ids)[3] == -1).all() and not out.weights[3].any()
    if score == "sigmoid":
        bias = torch.zeros(E, device="cuda")
        bias[::2] = float("-inf")
        out = fx.route_experts(x, k, bias=bias, score=score, renormalize=renorm, **kw)
        assert not ((out.ids >= 0) & (out.ids % 2 == 0)).any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_nan_and_infinity(score):
    """A NaN logit shows in its own token's weights (never a wrong index); other tokens are as
    without it."""
    g = gen(10)
    x = tied_logits(g, 20, 64)
    clean = fx.route_experts(x, 4, score=score)
    x[7, 13] = float("nan")
    x[9, 5] = float("inf")
    out = fx.route_experts(x, 4, score=score)
    keep = [i for i in range(20) if i not in (7, 9)]
    assert torch.equal(out.ids[keep], clean.ids[keep])
    assert torch.equal(out.weights[keep], clean.weights[keep])
    assert out.ids[7, 0] == 13 and torch.isnan(out.weights[7]).all()
    assert len(set(out.ids[7].tolist())) == 4
    assert out.ids[9, 0] == 5


def test_route_strided_rows_and_zero_sizes():
    g = gen(11)
    x = tied_logits(g, 19, 72).to(BF16)
    want = fx.route_experts(x, 5, score="sigmoid")
    for v in (strided(x, 8), strided(x, 3), shifted(x)):
        got = fx.route_experts(v, 5, score="sigmoid")
        assert torch.equal(got.ids, want.ids) and torch.equal(got.weights, want.weights)
    assert fx.route_experts(x[:0], 5).ids.shape == (0, 5)
    assert fx.route_experts(x, 0).ids.shape == (19, 0)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False),
                                          ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (33, 256, 8), (5, 31, 31), (70, 160, 6), (3, 1024, 32)])
def test_route_backward(T, E, k, score, renorm, dtype):
    g = gen(T + E)
    x = randn(g, T, E, dtype=dtype, scale=1.5)
    ids = fx.route_experts(x, k, score=score, renormalize=renorm).ids
    ids[T // 2, 0] = -1          # a slot without an expert
    ids[0, -1] = E + 3           # and one that names none of these
    dw = randn(g, T, k)
    dx = fx.route_experts_backward(dw, x, ids, score=score, renormalize=renorm, scale=1.25)
    want = ref.route_backward(np64(dw), np64(x), np64(ids), score == "sigmoid", renorm, 1.25)
    # the terms g_j and sum(p g) cancel: relative to the largest term, with p <= 1
    size = 1.25 * np.abs(np64(dw)).max(-1, keepdims=True) * 8
    close(dx, want, rounding(dtype, want) + 4 * U * np.abs(want) + WEIGHT_TOL * size, "dlogits")


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False),
                                          ("softmax", True), ("softmax", False)])
def test_route_backward_against_differences(score, renorm):
    g = gen(12)
    x, dw = randn(g, 4, 12), randn(g, 4, 3)
    ids = fx.route_experts(x, 3, score=score, renormalize=renorm).ids
    ids[2, 1] = -1
    dx = fx.route_experts_backward(dw, x, ids, score=score, renormalize=renorm, scale=0.5)
    check_differences(lambda v: (ref.route_weights(v, np64(ids), score == "sigmoid", renorm, 0.5)
                                 * np64(dw)).sum(), np64(x), np64(dx))


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("softmax", True), ("softmax", False)])
def test_route_backward_masked_rows(score, renorm):
    """Masked experts and tokens without any get zeros, not NaN; experts named twice add up."""
    g = gen(13)
    x = randn(g, 6, 16)
    x[1, :14] = float("-inf")
    x[2] = float("-inf")
    r = fx.route_experts(x, 4, score=score, renormalize=renorm)
    dx = fx.route_experts_backward(randn(g, 6, 4), x, r.ids, score=score, renormalize=renorm)
    assert torch.isfinite(dx).all() and not dx[2].any() and not dx[1, :14].any()
    twice = torch.tensor([[3, 3]], dtype=torch.int32, device="cuda")
    dw = torch.tensor([[0.5, 0.25]], device="cuda")
    got = fx.route_experts_backward(dw, x[:1], twice, score="sigmoid", renormalize=False)
    s = ref.sigmoid(np64(x[:1, 3]))
    close(got[:, 3], 0.75 * s * (1 - s), 1e-6, "an expert named twice")


@pytest.mark.parametrize("E,top_k", [(31, 8), (64, 1), (200, 8), (256, 20), (500, 8), (1024, 32)])
@pytest.mark.parametrize("spread", [3, 40, 5000, 1 << 20])
def test_route_order_of_near_ties(E, top_k, spread):
    """Logits a few steps of their last bit apart: a softmax without bias takes them in their
    order, equal ones by index, whatever the bits that an index displaces."""
    g = gen(E + spread)
    steps = torch.randint(0, spread, (300, E), generator=g, device="cuda").to(torch.int32)
    steps[200:] = -steps[200:]
    logits = (steps + 0x3F800000).view(torch.float32)  # from 1.0 on, and below
    got = np64(fx.route_experts(logits, top_k).ids)
    values = np64(logits)
    want = np.stack([np.lexsort((np.arange(E), -v))[:top_k] for v in values])
    assert np.array_equal(got, want)


# ---------------------------------------------------------------------------------------
# dispatch and combine
# ---------------------------------------------------------------------------------------
def random_ids(g, T, k, E, elsewhere=0.0):
    ids = torch.rand((T, max(E, k)), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    ids[ids >= E] = -1
    ids[torch.rand((T, k), generator=g, device="cuda") < elsewhere] = -1
    return ids


@pytest.mark.parametrize("T,k,E,H,cols,elsewhere", [
    (1, 1, 1, 16, 1, 0.0), (1, 8, 32, 7168, 1, 0.5), (3, 2, 8, 128, 1, 0.0), (129, 8, 256, 256, 2, 0.0),
    (511, 2, 16, 48, 1, 0.3), (512, 2, 16, 48, 0, 0.0), (513, 2, 16, 33, 1, 0.0),
    (2048, 1, 1024, 16, 1, 0.2), (2049, 1, 1024, 16, 1, 0.0), (300, 7, 9, 32, 1, 0.1),
    (9000, 8, 1024, 16, 1, 0.2), (70000, 2, 4, 16, 0, 0.5), (400, 8, 16, 24, 1, 0.2),
    (500, 6, 16, 12, 0, 0.0), (450, 5, 8, 6, 1, 0.3), (40, 2, 8, 1000, 1, 0.0), (2500, 2, 8, 1000, 1, 0.0), (4099, 1, 1, 16, 0, 0.0), (1500, 6, 60, 64, 3, 0.9), (5000, 8, 128, 16, 1, 0.1),
    (100, 32, 40, 80, 1, 0.0), (64, 4, 3, 1, 1, 0.0), (40, 8, 16, 100, 1, 1.0)])
def test_dispatch(T, k, E, H, cols, elsewhere):
    g = gen(T + E)
    x = torch.randint(0, 256, (T, H), generator=g, device="cuda").to(torch.uint8)
    scale = randn(g, T, cols) if cols > 1 else (randn(g, T) if cols else None)
    ids = random_ids(g, T, k, E, elsewhere)
    m, dest, source = ref.dispatch(np64(ids), E)
    poison = torch.full((T * k, H), 0x5A, dtype=torch.uint8, device="cuda")
    tail = tuple(scale.shape[1:]) if cols else ()
    out = fx.Dispatch(poison, torch.full((T * k, *tail), -7.0, device="cuda") if cols else None,
                      torch.full((E,), -1, device="cuda"),
                      torch.full((T, k), -9, dtype=torch.int32, device="cuda"))
    for _ in range(2):
        got = fx.moe_dispatch(x, scale, ids, E, out=out)
        assert got is out
        assert np.array_equal(np64(out.m_sizes), m)
        assert np.array_equal(np64(out.dest), dest)
        n = len(source)
        src = torch.from_numpy(source).cuda()
        assert torch.equal(out.x[:n], x[src])
        assert (out.x[n:] == 0x5A).all(), "rows past the last choice written"
        if cols:
            assert torch.equal(out.x_scale[:n], scale[src])
            assert (out.x_scale[n:] == -7.0).all()
    fresh = fx.moe_dispatch(x, scale, ids, E)
    assert torch.equal(fresh.x[:n], x[src]) and not fresh.x[n:].any()


@pytest.mark.parametrize("T,k,E,H,cols,elsewhere", [
    (2500, 1, 1000, 64, 1, 0.0), (2400, 8, 700, 32, 0, 0.9), (3000, 8, 256, 48, 2, 0.2),
    (20000, 8, 256, 33, 0, 0.1), (70001, 8, 40, 16, 1, 0.5), (16500, 10, 1024, 8, 0, 0.0)])
def test_dispatch_many_choices(T, k, E, H, cols, elsewhere):
    """Sorts of 8 and 16 CTAs, of a warp's choices at once and in several steps."""
    test_dispatch(T, k, E, H, cols, elsewhere)


def test_dispatch_of_rows_off_32_bytes():
    g = gen(77)
    ids = random_ids(g, 2100, 2, 9, 0.4)
    base = torch.randint(0, 256, (2100 * 64 + 16,), generator=g, device="cuda").to(torch.uint8)
    want = fx.moe_dispatch(base[:2100 * 64].view(2100, 64).clone(), None, ids, 9)
    x = base[16:].view(2100, 64)
    got = fx.moe_dispatch(x, None, ids, 9)
    n = int(got.m_sizes.sum())
    _, dest, source = ref.dispatch(np64(ids), 9)
    assert np.array_equal(np64(got.dest), dest) and torch.equal(got.dest, want.dest)
    assert torch.equal(got.x[:n], x[torch.from_numpy(source).cuda()])


def test_dispatch_foreign_ids_and_other_types():
    """Ids that name no expert here, of any value; rows of bf16; rows of odd bytes, unaligned."""
    g = gen(15)
    T, k, E = 90, 4, 12
    ids = torch.randint(-3, E + 3, (T, k), generator=g, device="cuda").to(torch.int32)
    ids[0] = torch.tensor([-2 ** 31, 2 ** 31 - 1, E, -1], dtype=torch.int32)
    m, dest, source = ref.dispatch(np.where((np64(ids) < 0) | (np64(ids) >= E), -1, np64(ids)), E)
    src = torch.from_numpy(source).cuda()
    for x in (randn(g, T, 56, dtype=BF16), randn(g, T, 9, dtype=BF16), randn(g, T, 64),
              shifted(randn(g, T, 64, dtype=FP16))):
        out = fx.moe_dispatch(x, None, ids, E)
        assert out.x_scale is None and np.array_equal(np64(out.m_sizes), m)
        assert np.array_equal(np64(out.dest), dest)
        assert torch.equal(out.x[:len(source)], x[src]) and not out.x[len(source):].any()


def test_dispatch_nothing():
    x = torch.zeros((0, 64), dtype=torch.uint8, device="cuda")
    out = fx.moe_dispatch(x, None, torch.zeros((0, 8), dtype=torch.int32, device="cuda"), 16)
    assert not out.m_sizes.any() and out.x.shape == (0, 64) and out.dest.shape == (0, 8)
    x = torch.zeros((5, 64), dtype=torch.uint8, device="cuda")
    out = fx.moe_dispatch(x, None, torch.zeros((5, 2), dtype=torch.int32, device="cuda"), 0)
    assert (out.dest == -1).all() and out.m_sizes.shape == (0,)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,k,E,H,elsewhere", [(1, 8, 16, 7168, 0.0), (5, 2, 4, 33, 0.3),
                                               (65, 8, 32, 1000, 0.5), (40, 32, 64, 256, 0.1),
                                               (3, 1, 2, 8, 0.0), (30, 6, 8, 4097, 1.0),
                                               (130, 8, 16, 64, 0.2), (21, 4, 8, 24, 0.0),
                                               (17, 3, 4, 1, 0.3), (11, 5, 9, 4104, 0.1)])
def test_combine(T, k, E, H, elsewhere, dtype):
    g = gen(T + H)
    ids = random_ids(g, T, k, E, elsewhere)
    _, dest, source = ref.dispatch(np64(ids), E)
    rows = randn(g, T * k, H, dtype=dtype)
    rows[len(source):] = float("nan")           # rows of no choice are not read
    dest = torch.from_numpy(dest).to(torch.int32).cuda()
    w = randn(g, T, k)
    w[dest < 0] = float("nan")                  # nor is the weight of a choice without a row
    for weights in (w, None):
        out = fx.moe_combine(rows, dest, weights)
        want, size = ref.combine(np64(rows), np64(dest), None if weights is None else np64(weights))
        close(out, want, rounding(dtype, want) + 34 * U * size, "out")


def test_combine_ignores_rows_outside():
    g = gen(18)
    rows, w = randn(g, 10, 64), randn(g, 4, 3)
    dest = torch.tensor([[0, 10, -1], [2 ** 31 - 1, -2 ** 31, 9], [3, 4, 5], [11, 12, -5]],
                        dtype=torch.int32, device="cuda")
    want, _ = ref.combine(np64(rows), np64(dest), np64(w))
    close(fx.moe_combine(rows, dest, w), want, 1e-6, "out")
    dout = randn(g, 4, 64)
    drows, dw = fx.moe_combine_backward(dout, rows, dest, w)
    assert not drows[[1, 2, 6, 7, 8]].any() and not dw[3].any() and dw[0, 1] == 0
    close(drows[9], np64(w)[1, 2] * np64(dout)[1], 1e-6, "drows")


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,k,E,H,elsewhere", [(1, 8, 16, 7168, 0.0), (5, 2, 4, 33, 0.3),
                                               (65, 8, 32, 1000, 0.5), (40, 32, 64, 256, 0.1),
                                               (3, 1, 2, 8, 0.0), (9, 6, 8, 4097, 1.0),
                                               (130, 8, 16, 64, 0.2), (21, 4, 8, 24, 0.0),
                                               (17, 3, 4, 1, 0.3), (11, 5, 9, 4104, 0.1)])
def test_combine_backward(T, k, E, H, elsewhere, dtype):
    g = gen(T + H + 1)
    ids = random_ids(g, T, k, E, elsewhere)
    _, dest, source = ref.dispatch(np64(ids), E)
    rows, dout, w = randn(g, T * k, H, dtype=dtype), randn(g, T, H, dtype=dtype), randn(g, T, k)
    drows, dw = fx.moe_combine_backward(dout, rows, torch.from_numpy(dest).to(torch.int32).cuda(), w)
    want_rows, want_w, size = np.zeros((T * k, H)), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if dest[t, j] >= 0:
                want_rows[dest[t, j]] = np64(w)[t, j] * np64(dout)[t]
                terms = np64(dout)[t] * np64(rows)[dest[t, j]]
                want_w[t, j], size[t, j] = terms.sum(), np.abs(terms).sum()
    close(drows, want_rows, rounding(dtype, want_rows) + U * np.abs(want_rows), "drows")
    # a thread's chain (16 columns at 512 threads and 7168 columns), the warp's 5, 16 warps
    close(dw, want_w, 48 * U * size, "dweights")


def test_combine_backward_against_differences():
    g = gen(20)
    rows, w, dout = randn(g, 6, 9), randn(g, 3, 2), randn(g, 3, 9)
    dest = torch.tensor([[4, 1], [0, -1], [5, 2]], dtype=torch.int32, device="cuda")
    drows, dw = fx.moe_combine_backward(dout, rows, dest, w)

    def loss(r, v):
        return (ref.combine(r, np64(dest), v)[0] * np64(dout)).sum()

    check_differences(lambda v: loss(v, np64(w)), np64(rows), np64(drows))
    check_differences(lambda v: loss(np64(rows), v), np64(w), np64(dw))


def test_dispatch_gradient_is_the_unweighted_combine():
    """<dispatch(x), r> = <x, combine(r)>: the two are transposes of each other."""
    g = gen(21)
    T, k, E, H = 50, 4, 8, 96
    ids = random_ids(g, T, k, E, 0.3)
    x = randn(g, T, H)
    packed = fx.moe_dispatch(x, None, ids, E)
    r = randn(g, T * k, H)
    left = (packed.x.double() * r.double()).sum()
    right = (x.double() * fx.moe_combine(r, packed.dest).double()).sum()
    assert abs(left - right) <= 1e-5 * abs(left) + 1e-3


# ---------------------------------------------------------------------------------------
# SwiGLU
# ---------------------------------------------------------------------------------------
# exp (2 ulp, and its argument's rounding), 1 + e, the division and two products
SWIGLU_REL = 16 * U


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("R,W,groupwise,checkpoint", [
    (1, 2048, False, False), (1, 128, True, True), (33, 2048, True, True), (5, 384, False, True),
    (3, 1, False, False), (17, 1000, False, False), (6, 1003, False, False), (40, 640, True, False),
    (3, 4224, True, True), (9, 3968, True, True), (70, 1920, True, False), (600, 256, True, True),
    (5, 16384, True, True), (5, 12288, False, False), (300, 125, False, False),
    (1001, 128, False, True), (41, 512, False, True), (37, 256, False, True), (3, 8208, False, False),
    (33, 48, False, False), (70, 1536, False, True), (9, 4104, False, False), (2, 8192, True, True), (2, 8320, True, True), (2, 32768, False, True),
    (1, 32767, False, False)])
def test_swiglu(R, W, groupwise, checkpoint, dtype):
    g = gen(R + W)
    x = randn(g, R, 2 * W, dtype=dtype, scale=2.0)
    out = fx.swiglu_quant(x, groupwise=groupwise, checkpoint=checkpoint)
    ref.check_codes(out.q, out.scale, ref.swiglu(np64(x)), ref.BLOCK if groupwise else W,
                    SWIGLU_REL, "q")
    if checkpoint:
        ref.check_codes(out.saved, out.saved_scale, np64(x), ref.BLOCK, 2 * U, "checkpoint")
    else:
        assert out.saved is None and out.saved_scale is None


def test_swiglu_strides_and_alignment():
    g = gen(22)
    R, W = 12, 256
    x = randn(g, R, 2 * W, dtype=BF16)
    want = fx.swiglu_quant(x, groupwise=True, checkpoint=True)
    for v in (strided(x, 16), strided(x, 5), shifted(x)):
        got = fx.swiglu_quant(v, groupwise=True, checkpoint=True)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    dy = randn(g, R, W, dtype=BF16)
    dx = fx.swiglu_quant_backward(dy, want.saved, want.saved_scale)
    for d, s in ((shifted(dy), want.saved), (dy, shifted(want.saved.view(torch.uint8)))):
        assert torch.equal(fx.swiglu_quant_backward(d, s, want.saved_scale), dx)
    assert torch.equal(fx.swiglu_quant_backward(dy, shifted(x)), fx.swiglu_quant_backward(dy, x))


def test_swiglu_extremes():
    """Zeros, gates far out on both sides, values past the fp32 product, NaN: each in its row."""
    W = 256
    x = torch.zeros(7, 2 * W, device="cuda")
    g = gen(23)
    x[1] = randn(g, 2 * W) * 1e-30
    x[2, :W] = -200.0
    x[2, W:] = 1.0
    x[3, :W] = 200.0
    x[3, W:] = randn(g, W)
    x[4] = randn(g, 2 * W)
    x[4, 5] = float("nan")
    x[5, 0], x[5, W] = 2.0 ** -70, 2.0 ** -9    # the one nonzero product is just above 2^-80
    x[6] = randn(g, 2 * W)
    for groupwise in (False, True):
        out = fx.swiglu_quant(x, groupwise=groupwise, checkpoint=True)
        fine = [0, 1, 2, 3, 5, 6]
        ref.check_codes(out.q[fine], out.scale[fine], ref.swiglu(np64(x[fine])),
                        ref.BLOCK if groupwise else W, SWIGLU_REL, "q")
        assert torch.isnan(out.scale[4].reshape(-1)[0]) and torch.isnan(out.saved_scale[4, 0])
        assert torch.isfinite(out.saved_scale[4, 1:]).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("R,W", [(1, 128), (1, 2048), (70, 384), (5, 4096), (3, 33), (4, 1000),
                                 (300, 125), (9, 3968), (130, 1), (3, 32768)])
def test_swiglu_backward(R, W, dtype):
    g = gen(R * W)
    x, dy = randn(g, R, 2 * W, dtype=dtype, scale=2.0), randn(g, R, W, dtype=dtype)
    kept = [(x, None, np64(x))]
    if W % ref.BLOCK == 0:
        out = fx.swiglu_quant(x, checkpoint=True)
        values = np64(out.saved).reshape(R, -1, ref.BLOCK) * np64(out.saved_scale)[..., None]
        kept.append((out.saved, out.saved_scale, values.reshape(R, 2 * W)))
    for saved, scale, values in kept:
        dx = fx.swiglu_quant_backward(dy, saved, scale)
        want = ref.swiglu_backward(np64(dy), values)
        gate, up = np.split(values, 2, axis=1)
        s = ref.sigmoid(gate)
        size = np.concatenate([np.abs(np64(dy) * up) * s * (1 + np.abs(gate)),
                               np.abs(np64(dy) * gate) * s], axis=1)
        close(dx, want, rounding(dtype, want) + 24 * U * size, "dx")


def test_swiglu_backward_against_differences():
    g = gen(25)
    x, dy = randn(g, 3, 10), randn(g, 3, 5)
    dx = fx.swiglu_quant_backward(dy, x)
    check_differences(lambda v: (ref.swiglu(v) * np64(dy)).sum(), np64(x), np64(dx))


def test_swiglu_backward_far_gates():
    x = torch.tensor([[-300.0, 300.0, 0.0, -88.0, 2.0, 3.0, 1.0, 1.0]], device="cuda")
    dy = torch.ones((1, 4), device="cuda")
    want = ref.swiglu_backward(np64(dy), np64(x))
    close(fx.swiglu_quant_backward(dy, x), want, 1e-6 * np.abs(want) + 1e-30, "dx")


# ---------------------------------------------------------------------------------------
# streams, graphs, long buffers, refusals
# ---------------------------------------------------------------------------------------
def moe_step(x, res, w, logits, E):
    n = fx.add_rms_norm_quant(x, w, res, want_y=True)
    r = fx.route_experts(logits, 4, score="sigmoid")
    d = fx.moe_dispatch(n.q, n.scale, r.ids, E)
    rows = d.x.to(BF16)
    return n, r, d, fx.moe_combine(rows, d.dest, r.weights)


def flat(v):
    return [t.view(torch.uint8) if t.dtype == E4M3 else t
            for part in v for t in (part if isinstance(part, tuple) else (part,)) if t is not None]


def test_side_stream_given_as_argument():
    g = gen(30)
    x, res, w = randn(g, 40, 512, dtype=BF16), randn(g, 40, 512, dtype=BF16), randn(g, 512, dtype=BF16)
    want = fx.add_rms_norm_quant(x, w, res, want_y=True, want_rstd=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = fx.add_rms_norm_quant(x, w, res, want_y=True, want_rstd=True, stream=stream)
        side.synchronize()
        for a, b in zip(flat(got), flat(want)):
            assert torch.equal(a, b)


def test_graph_capture_and_replay():
    g = gen(31)
    E = 16
    x, res, w = randn(g, 40, 512, dtype=BF16), randn(g, 40, 512, dtype=BF16), randn(g, 512, dtype=BF16)
    logits = randn(g, 40, E)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe_step(x, res, w, logits, E)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moe_step(x, res, w, logits, E)
    for seed in (32, 33):
        h = gen(seed)
        x.copy_(randn(h, 40, 512, dtype=BF16))
        logits.copy_(randn(h, 40, E))
        graph.replay()
        want = moe_step(x, res, w, logits, E)
        torch.cuda.synchronize()
        for a, b in zip(flat(got), flat(want)):
            assert torch.equal(a, b)


def test_back_to_back_calls_on_other_data():
    """Calls that nothing waits between, each on its own data, workspaces and outputs."""
    g = gen(34)
    E, cases = 32, []
    for T in (1, 64, 700):
        cases.append((randn(g, T, 256, dtype=BF16), randn(g, T, 256, dtype=BF16),
                      randn(g, 256, dtype=BF16), randn(g, T, E)))
    want = []
    for c in cases:
        want.append(moe_step(*c, E))
        torch.cuda.synchronize()
    got = [moe_step(*cases[i % 3], E) for i in range(12)]
    torch.cuda.synchronize()
    for i, v in enumerate(got):
        for a, b in zip(flat(v), flat(want[i % 3])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("op", ["norm", "dispatch", "combine", "swiglu"])
def test_offsets_past_32_bits(op):
    """Buffers of more than 2^32 bytes and 2^31 elements: the last rows are as on their own."""
    free = torch.cuda.mem_get_info()[0]
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    g = gen(35)
    if op == "norm":
        T, H = 270000, 8192
        x = torch.empty((T, H), dtype=BF16, device="cuda").fill_(0.5)
        x[-3:] = randn(g, 3, H, dtype=BF16)
        w = randn(g, H, dtype=BF16)
        out = fx.add_rms_norm_quant(x, w, x, want_y=True, want_rstd=True)
        small = fx.add_rms_norm_quant(x[-3:].clone(), w, x[-3:].clone(), want_y=True, want_rstd=True)
        for a, b in zip(flat(out), flat(small)):
            assert torch.equal(a[-3:], b)
        del out
        dx, _ = fx.add_rms_norm_quant_backward(x, x, w, torch.ones(T, device="cuda"), x)
        want, _ = fx.add_rms_norm_quant_backward(x[-3:].clone(), x[-3:].clone(), w,
                                                 torch.ones(3, device="cuda"), x[-3:].clone())
        assert torch.equal(dx[-3:], want)
    elif op in ("dispatch", "combine"):
        T, k, E, H = 70000, 8, 16, 8192
        ids = (torch.arange(T * k, device="cuda").reshape(T, k) % E).to(torch.int32)
        x = torch.randint(0, 200, (T, H), generator=g, device="cuda", dtype=torch.uint8)
        d = fx.moe_dispatch(x, None, ids, E)
        for t in (0, T // 2, T - 1):
            for j in range(k):
                assert torch.equal(d.x[int(d.dest[t, j])], x[t])
        assert int(d.dest.max()) == T * k - 1 and int(d.m_sizes.sum()) == T * k
        if op == "combine":
            dest = d.dest
            del d, x
            rows = torch.empty((T * k, H), dtype=BF16, device="cuda").fill_(1.0)
            at = dest[-1].long()
            rows[at] = randn(g, k, H, dtype=BF16)
            w = torch.rand((T, k), generator=g, device="cuda")
            want, size = ref.combine(np64(rows[at]), np.arange(k)[None], np64(w[-1:]))
            out = fx.moe_combine(rows, dest, w)
            close(out[-1:], want, rounding(BF16, want) + 34 * U * size, "out")
            drows, dw = fx.moe_combine_backward(out, rows, dest, w)
            close(drows[at], np64(w)[-1][:, None] * np64(out[-1:]),
                  2.0 ** -8 * np.abs(np64(w)[-1][:, None] * np64(out[-1:])), "drows")
    else:
        R, W = 140000, 8192
        x = torch.empty((R, 2 * W), dtype=BF16, device="cuda").fill_(0.5)
        x[-3:] = randn(g, 3, 2 * W, dtype=BF16)
        small = fx.swiglu_quant(x[-3:].clone(), groupwise=True, checkpoint=True)
        out = fx.swiglu_quant(x, groupwise=True, checkpoint=True)
        for a, b in zip(flat(out), flat(small)):
            assert torch.equal(a[-3:], b)
        dy = torch.ones((R, W), dtype=BF16, device="cuda")
        dx = fx.swiglu_quant_backward(dy, out.saved, out.saved_scale)
        assert torch.equal(dx[-3:], fx.swiglu_quant_backward(dy[-3:].clone(), small.saved,
                                                             small.saved_scale))


def test_refusals():
    """Wrong types, shapes, devices, strides and options raise before anything runs."""
    x = torch.zeros((4, 256), dtype=BF16, device="cuda")
    w = torch.ones(256, dtype=BF16, device="cuda")
    logits = torch.zeros((4, 16), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    norm, err = fx.add_rms_norm_quant, (TypeError, ValueError, fx.MslkbError)
    for call in (
            lambda: norm(x.cpu(), w), lambda: norm(x.double(), w), lambda: norm(x[0], w),
            lambda: norm(x.t(), w[:4]), lambda: norm(x, w[:128]), lambda: norm(x, w.half()),
            lambda: norm(x, w, x[:2]), lambda: norm(x, w, x.float()), lambda: norm(x, w, x.cpu()),
            lambda: norm(x, w, eps=0.0), lambda: norm(x, w, eps=float("nan")),
            lambda: norm(x[:, :100], w[:100], groupwise=True),
            lambda: norm(x, w, x.expand(4, 256)[:1].expand(4, 256)),
            lambda: norm(x, w, want_y=True, out=norm(x, w)),
            lambda: norm(x, w, out=(x, x)),
            lambda: norm(torch.zeros((1, 32776), dtype=BF16, device="cuda"),
                         torch.ones(32776, dtype=BF16, device="cuda")),
            lambda: fx.add_rms_norm_quant_backward(x, x, w, torch.ones(3, device="cuda")),
            lambda: fx.add_rms_norm_quant_backward(x, x[:, ::2], w, torch.ones(4, device="cuda")),
            lambda: fx.route_experts(logits, 17), lambda: fx.route_experts(logits, 2, score="relu"),
            lambda: fx.route_experts(logits, 2, num_groups=3),
            lambda: fx.route_experts(logits, 6, num_groups=4, topk_groups=1),
            lambda: fx.route_experts(logits, 2, num_groups=4, topk_groups=5),
            lambda: fx.route_experts(logits, 2, num_groups=4, topk_groups=2, group_top=3),
            lambda: fx.route_experts(logits, 2, bias=torch.zeros(16, device="cuda").half()),
            lambda: fx.route_experts(torch.zeros((2, 1025), device="cuda"), 2),
            lambda: fx.route_experts(torch.zeros((2, 64), device="cuda"), 33),
            lambda: fx.route_experts_backward(logits[:, :2], logits, ids),
            lambda: fx.route_experts_backward(torch.zeros((4, 2), device="cuda"), logits, ids.long()),
            lambda: fx.moe_dispatch(x, None, ids.long(), 4), lambda: fx.moe_dispatch(x, None, ids[:3], 4),
            lambda: fx.moe_dispatch(x, torch.ones(3, device="cuda"), ids, 4),
            lambda: fx.moe_dispatch(x, None, ids, 1025), lambda: fx.moe_dispatch(x.cpu(), None, ids, 4),
            lambda: fx.moe_dispatch(x[:, ::2], None, ids, 4),
            lambda: fx.moe_combine(x, ids, torch.ones((4, 3), device="cuda")),
            lambda: fx.moe_combine(x.double(), ids), lambda: fx.moe_combine(x, ids.cpu()),
            lambda: fx.moe_combine_backward(x, x[:, :128], ids, torch.ones((4, 2), device="cuda")),
            lambda: fx.swiglu_quant(x[:, :255]), lambda: fx.swiglu_quant(x[:, :200], checkpoint=True),
            lambda: fx.swiglu_quant(x[:, :200], groupwise=True), lambda: fx.swiglu_quant(x.to(E4M3)),
            lambda: fx.swiglu_quant_backward(x[:, :128].contiguous(), x.float()),
            lambda: fx.swiglu_quant_backward(x[:, :128].contiguous(), x.to(E4M3),
                                             torch.ones((4, 1), device="cuda"))):
        with pytest.raises(err):
            call()
    torch.cuda.synchronize()
    assert fx.device_status() == 0
