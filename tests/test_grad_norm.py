"""The norm of a list of gradients and their clipping on the GPU, against 64 bits: one element to
many tensors, types mixed, sizes and addresses of every alignment, values at the ends of the
types' ranges, values that are not numbers, in place, streams, graphs, refusals.

Tolerances.  u = 2^-24.  Squares of a 16-byte vector and of up to four vectors are summed in fp32
(at most 33 roundings, each of at most u of the sum, all terms positive), everything above that
without loss or in 64 bits; the root halves a relative error and is rounded once: 18 u.  A clipped
gradient is g * scale with scale = max_norm / (norm + eps), two fp32 roundings besides the
norm's error, and the product's own: (18 + 3) u, and then the rounding to its type.
"""
import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import U, close, np64, rounding

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, FP16, FP32]
NAN, INF = float("nan"), float("inf")


def stream():
    """A stream of the pool that holds those of high priority: the ordinary pool's 32 go round, and
    tests that count the workspaces kept by stream take theirs from it."""
    return torch.cuda.Stream(priority=-1)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    fxbuild.build()
    fx.lib()


def randn(seed, *shape, dtype=FP32, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def grads_of(sizes, types=TYPES, seed=0, scale=0.01):
    return [randn(seed + i, n, dtype=types[i % len(types)], scale=scale * (1 + i % 7))
            for i, n in enumerate(sizes)]


def norm64(grads, inf=False):
    v = [np64(g).reshape(-1) for g in grads if g.numel()]
    if not v:
        return 0.0
    return max(np.abs(x).max() for x in v) if inf else np.sqrt(sum((x * x).sum() for x in v))


def check_norm(got, grads, inf=False):
    want = norm64(grads, inf)
    assert got.dtype == FP32 and got.numel() == 1
    assert abs(got.item() - want) <= (0 if inf else 18 * U * want), (got.item(), want)


def check_clip(got, grads, before, max_norm, eps=1e-6, inf=False):
    norm = norm64(before, inf)
    scale = min(1.0, max_norm / (norm + eps))
    for i, (g, b) in enumerate(zip(got, before)):
        want = np64(b) * scale
        close(np64(g), want, 21 * U * np.abs(want) + rounding(g.dtype, want), f"tensor {i}")


LISTS = [[1], [7], [0], [], [5, 0, 3], [1024] * 3, [4096, 1, 65537, 2, 33], [1 << 20],
         [3_000_001, 17], list(range(1, 70)), [129] * 300, [2000] * 1500, [70_001, 1_000_003, 64]]


@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("types", [[BF16], [FP16], [FP32], TYPES])
def test_lists(types, inf):
    for sizes in LISTS:
        grads = grads_of(sizes, types)
        kind = INF if inf else 2.0
        check_norm(fx.grad_norm(grads, norm_type=kind), grads, inf)
        norm = norm64(grads, inf)
        for max_norm in (0.37 * norm, 2.0 * norm + 1.0):
            r = fx.clip_grad_norm(grads, max_norm, norm_type=kind)
            check_norm(r.norm, grads, inf)
            check_clip(r.grads, grads, grads, max_norm, inf=inf)


@pytest.mark.parametrize("types", [[BF16], [FP32], TYPES])
def test_in_place(types):
    for sizes in ([1], [40, 0, 9000], [1_000_003, 70_000], [500] * 400):
        grads = grads_of(sizes, types)
        before = [g.clone() for g in grads]
        norm = torch.zeros((), device="cuda")
        max_norm = 0.5 * norm64(grads)
        r = fx.clip_grad_norm(grads, max_norm, out=(norm, grads))
        assert r.norm is norm and r.grads is grads
        check_norm(norm, before)
        check_clip(grads, grads, before, max_norm)
        # within the bound: nothing changes
        now = [g.clone() for g in grads]
        fx.clip_grad_norm(grads, 2 * max_norm + 1, out=(norm, grads))
        assert all(torch.equal(a, b) for a, b in zip(grads, now))


@pytest.mark.parametrize("dtype", TYPES)
def test_alignments(dtype):
    """Every offset of an element in a 16-byte line, for the gradient and for the result."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    for n in (3, per, 5 * per + 1, 4099, 200_001):
        for a in range(per):
            g = torch.zeros(n + per, dtype=dtype, device="cuda")[a:a + n]
            g.copy_(randn(a, n, dtype=dtype))
            for b in {a, 0, per - 1}:
                whole = torch.full((n + 2 * per,), 3.0, dtype=dtype, device="cuda")
                o = whole[b:b + n]
                norm = torch.zeros(1, device="cuda")
                max_norm = 0.3 * norm64([g])
                fx.clip_grad_norm([g], max_norm, out=(norm, [o]))
                check_norm(norm, [g])
                check_clip([o], [g], [g], max_norm)
                assert (whole[:b] == 3).all() and (whole[b + n:] == 3).all()


def test_dense_in_any_order():
    g = [randn(1, 40, 30).t(), randn(2, 2, 3, 4).permute(2, 0, 1), randn(3, 5, 7)]
    r = fx.clip_grad_norm(g, 1.0)
    check_norm(r.norm, g)
    check_clip(r.grads, g, g, 1.0)
    assert all(a.stride() == b.stride() for a, b in zip(r.grads, g))


@pytest.mark.parametrize("value", [2.0 ** 127, 1e30, 1.5 * 2.0 ** 50, 2.0 ** -50, 1e-20,
                                   2.0 ** -126, 2.0 ** -149])
@pytest.mark.parametrize("n", [1, 3, 1000, 300_000])
def test_ends_of_the_range(value, n):
    """Squares of such values leave fp32; their norm does not (2^127: from four on it does)."""
    g = torch.full((n,), value, device="cuda")
    want = np.sqrt(n) * np64(g[:1])[0]
    got = fx.grad_norm([g]).item()
    if want >= 2.0 ** 128:
        assert got == INF
    else:
        assert abs(got - want) <= max(18 * U * want, 2.0 ** -150)
    # beside ordinary ones, in one tensor and in another
    both = torch.cat([g, randn(1, 1000)])
    if value < 1e30:
        check_norm(fx.grad_norm([both, randn(2, 77)]), [both, randn(2, 77)])


def test_long_runs_of_equal_values():
    for dtype, value in ((BF16, 1.0078125), (FP32, 1 / 3)):
        g = torch.full((100_000_000,), value, dtype=dtype, device="cuda")
        want = 1e4 * np64(g[:1])[0]
        assert abs(fx.grad_norm([g]).item() - want) <= 18 * U * want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes", [[100, 3], [2_000_000, 70]])
def test_not_numbers(dtype, sizes):
    for at in (0, sizes[0] // 2, sizes[0] - 1):
        for inf in (False, True):
            kind = INF if inf else 2.0
            grads = grads_of(sizes, [dtype])
            grads[0][at] = -INF
            r = fx.clip_grad_norm(grads, 1.0, norm_type=kind)
            assert r.norm.item() == INF          # scale 0: infinity * 0 is not a number
            assert torch.isnan(r.grads[0][at]) and torch.isnan(r.grads[0]).sum() == 1
            assert not r.grads[1].any()
            grads[0][at] = NAN
            r = fx.clip_grad_norm(grads, 1.0, norm_type=kind)
            assert torch.isnan(r.norm) and all(torch.isnan(g).all() for g in r.grads)
            assert torch.isnan(fx.grad_norm(grads, norm_type=kind))


def test_zero_and_unbounded():
    grads = [torch.zeros(1000, device="cuda"), torch.zeros(3, dtype=BF16, device="cuda")]
    r = fx.clip_grad_norm(grads, 1.0)
    assert r.norm.item() == 0 and not any(g.any() for g in r.grads)
    grads = grads_of([1000, 70_000])
    r = fx.clip_grad_norm(grads, INF)
    assert all(torch.equal(a, b) for a, b in zip(r.grads, grads))
    r = fx.clip_grad_norm(grads, 0.0)
    assert not any(g.any() for g in r.grads)


def test_offsets_past_32_bits():
    n = 2 ** 31 + 12345
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-5:] = 2.0
    g[2 ** 31 - 3] = 1.0
    r = fx.clip_grad_norm([g], 1.0)
    want = np.sqrt(21.0)
    assert abs(r.norm.item() - want) <= 18 * U * want
    scaled = np64(torch.tensor([2.0 / (want + 1e-6)]).to(BF16))
    close(np64(r.grads[0][-5:]), np.full(5, scaled[0]), rounding(BF16, scaled), "last")
    assert int((r.grads[0] != 0).sum()) == 6


def test_bits_do_not_change():
    grads = grads_of([3_000_001, 70, 1_000_000] + [999] * 100)
    first = fx.grad_norm(grads)
    assert all(torch.equal(fx.grad_norm(grads), first) for _ in range(10))


def test_small_tensors_beside_large_ones():
    """Many small tensors in one CTA's run, before, between and behind large ones."""
    for types in ([BF16], [FP32], TYPES):
        sizes = ([1 + 37 * i for i in range(120)] + [3_000_001] +
                 [8192, 8191, 4097, 2048, 2049] * 8 + [5_000_000] + [7168] * 60)
        grads = grads_of(sizes, types)
        r = fx.clip_grad_norm(grads, 0.25)
        check_norm(r.norm, grads)
        check_clip(r.grads, grads, grads, 0.25)
        held = [g.clone() for g in grads]
        fx.clip_grad_norm(held, 0.25, out=(torch.zeros((), device="cuda"), held))
        assert all(torch.equal(a, b) for a, b in zip(held, r.grads))
        assert torch.equal(fx.grad_norm(grads), r.norm)


def test_streams_and_graphs():
    """Two graphs of different lists, replayed with new values side by side."""
    runs = []
    for sizes in ([3_000_001, 17, 900], [300, 40]):
        grads = grads_of(sizes)
        out = (torch.zeros((), device="cuda"), [torch.zeros_like(g) for g in grads])
        only = torch.zeros((), device="cuda")
        side = stream()
        torch.cuda.synchronize()
        fx.clip_grad_norm(grads, 0.25, out=out, stream=side)
        fx.grad_norm(grads, out=only, stream=side.cuda_stream)
        side.synchronize()
        check_norm(only, grads)
        check_clip(out[1], grads, grads, 0.25)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fx.clip_grad_norm(grads, 0.25, out=out)
            fx.grad_norm(grads, out=only)
        runs.append((graph, grads, out, only, stream()))
    for i, (_, grads, *_) in enumerate(runs):
        for j, g in enumerate(grads):
            g.copy_(randn(100 + 10 * i + j, *g.shape))
    torch.cuda.synchronize()
    for _ in range(4):
        for graph, *_, s in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, grads, out, only, _ in runs:
        check_norm(out[0], grads)
        check_norm(only, grads)
        check_clip(out[1], grads, grads, 0.25)


def test_refusals():
    g = [randn(1, 100), randn(2, 50, dtype=BF16)]
    norm = torch.zeros((), device="cuda")
    like = [torch.zeros_like(v) for v in g]
    flat = torch.zeros(300, device="cuda")
    bad = [
        (TypeError, lambda: fx.grad_norm(g[0])),
        (TypeError, lambda: fx.grad_norm([None])),
        (TypeError, lambda: fx.grad_norm([g[0].double()])),
        (ValueError, lambda: fx.grad_norm([g[0].cpu()])),
        (ValueError, lambda: fx.grad_norm([g[0][::2]])),
        (ValueError, lambda: fx.grad_norm([g[0].expand(3, 100)])),
        (ValueError, lambda: fx.grad_norm(g, norm_type=1)),
        (TypeError, lambda: fx.grad_norm(g, out=norm.double())),
        (ValueError, lambda: fx.grad_norm(g, out=torch.zeros(2, device="cuda"))),
        (ValueError, lambda: fx.grad_norm(g, out=torch.zeros(()))),
        (fx.MslkbError, lambda: fx.clip_grad_norm(g, -1.0)),
        (fx.MslkbError, lambda: fx.clip_grad_norm(g, NAN)),
        (fx.MslkbError, lambda: fx.clip_grad_norm(g, 1.0, eps=-1.0)),
        (fx.MslkbError, lambda: fx.clip_grad_norm(g, 1.0, eps=INF)),
        (TypeError, lambda: fx.clip_grad_norm(g, 1.0, out=norm)),
        (TypeError, lambda: fx.clip_grad_norm(g, 1.0, out=(norm, None))),
        (ValueError, lambda: fx.clip_grad_norm(g, 1.0, out=(norm, like[:1]))),
        (TypeError, lambda: fx.clip_grad_norm(g, 1.0, out=(norm, [like[0], like[1].half()]))),
        (ValueError, lambda: fx.clip_grad_norm(g, 1.0, out=(norm, [like[0][:99], like[1]]))),
        # results over each other, over another gradient, the same gradient twice in place
        (fx.MslkbError, lambda: fx.clip_grad_norm(
            [g[0], g[0]], 1.0, out=(norm, [flat[:100], flat[99:199]]))),
        (fx.MslkbError, lambda: fx.clip_grad_norm(
            [flat[:100], flat[100:200]], 1.0, out=(norm, [flat[100:200], flat[200:300]]))),
        (fx.MslkbError, lambda: fx.clip_grad_norm(
            [flat[:100], flat[:100]], 1.0, out=(norm, [flat[:100], flat[:100]]))),
        (fx.MslkbError, lambda: fx.clip_grad_norm([flat[:100]], 1.0, out=(norm, [flat[1:101]]))),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was taken")
    # the same gradient twice is fine where it is only read
    r = fx.clip_grad_norm([g[0], g[0]], 1.0)
    check_norm(r.norm, [g[0], g[0]])
