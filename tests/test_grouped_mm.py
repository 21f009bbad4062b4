"""The products by expert in 16 bits on the GPU against plain 64-bit forms: the product, the
product with the matrices turned (its input's gradient) and the weights' gradient; ragged and odd
sizes, experts without rows, strides and alignments, values that are not numbers in rows and
columns that do not belong, streams, graphs, long offsets, refusals.

Tolerances.  The products of two bf16 or fp16 numbers are exact in fp32 and the sum of n of them
is made in fp32, in steps that lose at most 2^-23 of what has been summed (one unit in the last
place, whichever way a step rounds): n * 2^-23 * sum |x w|.  The result is rounded once more.
"""
import numpy as np
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import close, np64, rounding

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
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


@pytest.fixture(autouse=True)
def _status():
    fx.device_status()
    yield
    assert fx.device_status() == 0


def randn(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def sizes(counts):
    return torch.tensor(counts, dtype=torch.int64, device="cuda")


def shifted(t):
    """The same values one element into a buffer: aligned for the element type only."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    b[1:] = t.reshape(-1)
    return b[1:].view(t.shape)


def strided(t, extra):
    """The same rows as slices of rows that are `extra` elements longer and hold NaN there."""
    b = torch.full((t.shape[0], t.shape[1] + extra), NAN, dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


def bounds(counts):
    ends = np.cumsum(counts)
    return list(zip(ends - counts, ends))


def off(n, magnitudes, want, dtype):
    """Tolerance: see above."""
    return n * 2.0 ** -23 * magnitudes + rounding(dtype, want)


def check_mm(out, x, w, counts, transposed, what="out"):
    x, w = np64(x), np64(w)
    for g, (a, b) in enumerate(bounds(counts)):
        m = w[g] if transposed else w[g].T
        want = x[a:b] @ m
        close(np64(out[a:b]), want, off(x.shape[1], np.abs(x[a:b]) @ np.abs(m), want, out.dtype),
              f"{what}, expert {g}")


def check_grad(dw, dy, x, counts, add=None, what="dw"):
    dy, x = np64(dy), np64(x)
    add = None if add is None else np64(add)
    for g, (a, b) in enumerate(bounds(counts)):
        want, mag = dy[a:b].T @ x[a:b], np.abs(dy[a:b]).T @ np.abs(x[a:b])
        if add is not None:
            want, mag = want + add[g], mag + np.abs(add[g])
        close(np64(dw[g]), want, off(b - a + 1, mag, want, dw.dtype), f"{what}, expert {g}")


COUNTS = [[1], [0, 1, 0], [300, 0, 5, 129, 1], [16, 16, 16, 16], [3, 17, 0, 64, 2, 0],
          [257, 255, 31], [700]]
SHAPES = [(64, 64), (8, 8), (256, 512), (136, 200), (1000, 1001), (333, 77), (1, 1), (1536, 72)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_mm(shape, transposed, dtype):
    n, k = shape
    for i, counts in enumerate(COUNTS):
        x = randn(i, sum(counts), k, dtype=dtype)
        w = randn(100 + i, len(counts), *((k, n) if transposed else (n, k)), dtype=dtype)
        out = fx.grouped_mm(x, w, sizes(counts), transposed=transposed)
        check_mm(out, x, w, counts, transposed, f"counts {counts}")


@pytest.mark.parametrize("dtype,grad", [(BF16, FP32), (BF16, BF16), (FP16, FP16), (FP16, FP32)])
@pytest.mark.parametrize("shape", SHAPES)
def test_weight_grad(shape, dtype, grad):
    n, k = shape
    for i, counts in enumerate(COUNTS):
        dy, x = randn(i, sum(counts), n, dtype=dtype), randn(50 + i, sum(counts), k, dtype=dtype)
        add = randn(99, len(counts), n, k, dtype=grad) if i % 2 else None
        dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=add, dtype=grad)
        assert dw.dtype == grad
        check_grad(dw, dy, x, counts, add, f"counts {counts}")


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("counts", [[1300, 40, 0, 3], [5, 2049, 7, 300, 0, 2], [1024] * 3,
                                    [4000, 1], [513] * 9])
@pytest.mark.parametrize("shape", [(200, 264), (512, 512), (77, 130)])
def test_weight_grad_many_rows(shape, counts, add):
    """Experts with more rows than the tensor core sums at a time, beside others with few; fp32
    sums are made 512 rows at a time, so the lost bits do not grow with the rows: 512 * 2^-23 of
    the magnitudes, and a rounding for each of the sums of 512."""
    n, k = shape
    m = sum(counts)
    dy, x = randn(1, m, n), randn(2, m, k)
    for grad in (FP32, BF16):
        before = randn(3, len(counts), n, k, dtype=grad) if add else None
        dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=before, dtype=grad)
        check_grad(dw, dy, x, counts, before)
        if grad is FP32:
            for g, (a, b) in enumerate(bounds(counts)):
                want, mag = np64(dy[a:b]).T @ np64(x[a:b]), np.abs(np64(dy[a:b])).T @ np.abs(
                    np64(x[a:b]))
                if add:
                    want, mag = want + np64(before[g]), mag + np.abs(np64(before[g]))
                close(np64(dw[g]), want, off(512 + (b - a) // 512 + 2, mag, want, FP32),
                      f"expert {g}")


def test_weight_grad_added_by_few_experts_rows():
    """What is added where most experts have few rows and two have many, in place as well."""
    counts = [2000, 0, 7, 1041] + [16] * 30
    n, k = 512, 776
    m = sum(counts)
    dy, x = randn(1, m, n), randn(2, m, k)
    for grad in (FP32, BF16):
        before = randn(3, len(counts), n, k, dtype=grad)
        dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=before)
        check_grad(dw, dy, x, counts, before)
        held = before.clone()
        assert fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=held, out=held) is held
        assert torch.equal(held, dw)


def test_weight_grad_error_does_not_grow():
    """Sums of 64 to 16384 rows of normal values, as 2-norms: half of the last place that the
    tensor core loses in each of 512 / 16 steps, downwards, is 32 * 2^-24 at the most."""
    for rows in (64, 1024, 4096, 16384):
        for experts in (1, 40):
            m = rows * experts
            dy, x = randn(rows, m, 64), randn(rows + 1, m, 128)
            dw = fx.grouped_mm_weight_grad(dy, x, sizes([rows] * experts))
            want = dy[-rows:].double().t() @ x[-rows:].double()
            rel = ((dw[-1].double() - want).norm() / want.norm()).item()
            assert rel <= 32 * 2.0 ** -24, (rows, experts, rel)


def test_weight_grad_in_place():
    counts = [40, 0, 9]
    dy, x = randn(1, 49, 128), randn(2, 49, 256)
    for grad in (FP32, BF16):
        add = randn(3, 3, 128, 256, dtype=grad)
        dw = add.clone()
        assert fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=dw, out=dw) is dw
        check_grad(dw, dy, x, counts, add)
        assert torch.equal(dw[1], add[1])


@pytest.mark.parametrize("make", [shifted, lambda t: strided(t, 8), lambda t: strided(t, 5),
                                  lambda t: strided(t, 64)])
def test_strides_and_alignment(make):
    counts = [70, 3, 200]
    m = sum(counts)
    x, dy = randn(1, m, 192), randn(2, m, 128)
    w = randn(3, 3, 128, 192)
    out = fx.grouped_mm(make(x), w, sizes(counts))
    check_mm(out, x, w, counts, False)
    dx = fx.grouped_mm(make(dy), w, sizes(counts), transposed=True)
    check_mm(dx, dy, w, counts, True)
    dw = fx.grouped_mm_weight_grad(make(dy), make(x), sizes(counts))
    check_grad(dw, dy, x, counts)


def test_outputs_and_weights_off_16_bytes():
    counts = [33, 90]
    x, w, dy = randn(1, 123, 64), randn(2, 2, 72, 64), randn(3, 123, 72)
    out = shifted(torch.zeros((123, 72), dtype=BF16, device="cuda"))
    fx.grouped_mm(x, shifted(w), sizes(counts), out=out)
    check_mm(out, x, w, counts, False)
    for grad in (FP32, BF16):
        dw = shifted(torch.zeros((2, 72, 64), dtype=grad, device="cuda"))
        fx.grouped_mm_weight_grad(dy, x, sizes(counts), out=dw)
        check_grad(dw, dy, x, counts)


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("k", [64, 200, 77])
def test_values_that_do_not_belong(k, bad):
    """Not-a-number in an expert's rows stays with its rows; in rows past the last expert's and in
    an expert without rows it is not seen."""
    counts, n, spare = [5, 0, 130, 7], 136, 21
    m = sum(counts)
    x = torch.full((m + spare, k), bad, dtype=BF16, device="cuda")
    dy = torch.full((m + spare, n), bad, dtype=BF16, device="cuda")
    x[:m], dy[:m] = randn(1, m, k), randn(2, m, n)
    x[5:135], dy[5:135] = bad, bad           # all of expert 2
    w = randn(3, 4, n, k)
    w[1] = bad
    ms = sizes(counts)
    out = torch.full((m + spare, n), 7.0, dtype=BF16, device="cuda")
    fx.grouped_mm(x, w, ms, out=out)
    assert (out[m:] == 7.0).all()
    assert not torch.isfinite(out[5:135].float()).any()
    rest = [5, 0, 0, 7]
    keep = torch.cat([torch.arange(5), torch.arange(135, 142)]).cuda()
    check_mm(out[keep], x[keep], torch.where(torch.isfinite(w), w, 0), rest, False)
    dx = fx.grouped_mm(dy, w, ms, transposed=True)
    assert (dx[m:] == 0).all()
    check_mm(dx[keep], dy[keep], torch.where(torch.isfinite(w), w, 0), rest, True)
    dw = fx.grouped_mm_weight_grad(dy, x, ms)
    assert not torch.isfinite(dw[2]).any()
    dw[2] = 0
    check_grad(dw, dy[keep], x[keep], rest)


def test_one_bad_element():
    """A single NaN reaches exactly the sums that it is part of."""
    counts = [20, 30]
    x, w, dy = randn(1, 50, 96), randn(2, 2, 80, 96), randn(3, 50, 80)
    x[22, 17] = NAN
    out = fx.grouped_mm(x, w, sizes(counts))
    want = torch.zeros(50, 80, dtype=torch.bool, device="cuda")
    want[22] = True
    assert torch.equal(torch.isnan(out), want)
    dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts))
    want = torch.zeros(2, 80, 96, dtype=torch.bool, device="cuda")
    want[1, :, 17] = True
    assert torch.equal(torch.isnan(dw), want)


def test_nothing_to_sum():
    ms = sizes([3, 0])
    x, w = torch.empty((4, 0), dtype=BF16, device="cuda"), torch.empty((2, 72, 0), dtype=BF16,
                                                                         device="cuda")
    out = torch.full((4, 72), 5.0, dtype=BF16, device="cuda")
    fx.grouped_mm(x, w, ms, out=out)
    assert (out[:3] == 0).all() and (out[3] == 5).all()
    none = torch.empty((0, 64), dtype=BF16, device="cuda")
    add = randn(1, 2, 64, 64, dtype=FP32)
    assert torch.equal(fx.grouped_mm_weight_grad(none, none, sizes([0, 0]), add=add), add)
    assert (fx.grouped_mm_weight_grad(none, none, sizes([0, 0])) == 0).all()
    assert fx.grouped_mm(none, randn(2, 2, 8, 64), sizes([0, 0])).shape == (0, 8)
    assert fx.grouped_mm_weight_grad(none, none[:, :0], sizes([0, 0])).shape == (2, 64, 0)
    assert fx.grouped_mm(x[:, :0], randn(1, 0, 8, 0), sizes([])).shape == (4, 8)


def test_many_experts():
    """The most experts there may be, most of them without rows."""
    g = 1024
    counts = [(i * 7919) % 5 if i % 3 == 0 else 0 for i in range(g)]
    m = sum(counts)
    x, w, dy = randn(1, m, 32), randn(2, g, 40, 32), randn(3, m, 40)
    check_mm(fx.grouped_mm(x, w, sizes(counts)), x, w, counts, False)
    check_mm(fx.grouped_mm(dy, w, sizes(counts), transposed=True), dy, w, counts, True)
    check_grad(fx.grouped_mm_weight_grad(dy, x, sizes(counts)), dy, x, counts)


def test_counts_past_the_rows_are_clamped():
    x, w, dy = randn(1, 40, 64), randn(2, 3, 32, 64), randn(3, 40, 32)
    ms = sizes([30, -4, 1 << 40])
    for call in (lambda: check_mm(fx.grouped_mm(x, w, ms), x, w, [30, 0, 10], False),
                 lambda: check_grad(fx.grouped_mm_weight_grad(dy, x, ms), dy, x, [30, 0, 10])):
        call()
        assert fx.device_status() == fx.MSLKB_DEV_MSIZES_CLAMPED


def test_bits_do_not_change():
    counts = [100, 0, 413, 55]
    m = sum(counts)
    x, w, dy = randn(1, m, 1024), randn(2, 4, 512, 1024), randn(3, m, 512)
    ms = sizes(counts)
    first = (fx.grouped_mm(x, w, ms), fx.grouped_mm(dy, w, ms, transposed=True),
             fx.grouped_mm_weight_grad(dy, x, ms))
    for _ in range(5):
        again = (fx.grouped_mm(x, w, ms), fx.grouped_mm(dy, w, ms, transposed=True),
                 fx.grouped_mm_weight_grad(dy, x, ms))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_streams():
    counts = [37, 0, 91]
    x, w, dy = randn(1, 128, 256), randn(2, 3, 192, 256), randn(3, 128, 192)
    ms = sizes(counts)
    torch.cuda.synchronize()
    side = stream()
    out = fx.grouped_mm(x, w, ms, stream=side)
    dw = fx.grouped_mm_weight_grad(dy, x, ms, stream=side.cuda_stream)
    with torch.cuda.stream(side):
        dx = fx.grouped_mm(dy, w, ms, transposed=True)
    side.synchronize()
    check_mm(out, x, w, counts, False)
    check_mm(dx, dy, w, counts, True)
    check_grad(dw, dy, x, counts)


def test_two_graphs_at_once():
    """Captured once, replayed with other values and other counts, two of them side by side."""
    runs = []
    for i in range(2):
        x, w, dy = randn(i, 150, 256), randn(10 + i, 3, 192, 256), randn(20 + i, 150, 192)
        ms = sizes([50, 50, 50])
        out, dx = torch.zeros_like(dy), torch.zeros_like(x)
        dw = torch.zeros((3, 192, 256), device="cuda")

        def calls():
            fx.grouped_mm(x, w, ms, out=out)
            fx.grouped_mm(dy, w, ms, transposed=True, out=dx)
            fx.grouped_mm_weight_grad(dy, x, ms, out=dw)
        calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        runs.append((graph, x, w, dy, ms, out, dx, dw))
    counts = [[0, 149, 1], [77, 0, 73]]
    for (_, x, _, _, ms, *_), c in zip(runs, counts):
        ms.copy_(sizes(c))
        x.copy_(randn(40 + c[1], 150, 256))
    torch.cuda.synchronize()
    streams = [stream(), stream()]
    for _ in range(3):
        for (graph, *_), s in zip(runs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, x, w, dy, _, out, dx, dw), c in zip(runs, counts):
        check_mm(out, x, w, c, False)
        check_mm(dx, dy, w, c, True)
        check_grad(dw, dy, x, c)


def test_offsets_past_32_bits():
    """Outputs of over 2^31 elements: the last rows and the last expert."""
    rows, n, k = 270_000, 8192, 64
    x, w = randn(1, rows, k), randn(2, 2, n, k)
    counts = [rows - 9, 9]
    out = fx.grouped_mm(x, w, sizes(counts))
    assert out.numel() > 2 ** 31
    want = np64(x[-9:]) @ np64(w[1]).T
    close(np64(out[-9:]), want, off(k, np.abs(np64(x[-9:])) @ np.abs(np64(w[1])).T, want, BF16),
          "last rows")
    at = rows - 20
    want = np64(x[at:at + 11]) @ np64(w[0]).T
    close(np64(out[at:at + 11]), want,
          off(k, np.abs(np64(x[at:at + 11])) @ np.abs(np64(w[0])).T, want, BF16), "expert 0")
    del out
    g, n, k = 40, 8192, 8192
    counts = [0] * 38 + [3, 5]
    dy, x = randn(3, 8, n), randn(4, 8, k)
    dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts), dtype=BF16)
    assert dw.numel() > 2 ** 31
    assert not dw[:38].any()
    for e, (a, b) in ((38, (0, 3)), (39, (3, 8))):
        want = np64(dy[a:b]).T @ np64(x[a:b])
        close(np64(dw[e]), want, off(6, np.abs(np64(dy[a:b])).T @ np.abs(np64(x[a:b])), want, BF16),
              f"expert {e}")


def test_gradients_against_differences():
    """d/dt of sum(g * mm(x + t u, w + t v)) at 0: the function is quadratic in t, so the central
    difference in 64 bits is exact, and the kernels' gradients are the formulas'."""
    counts, n, k = [13, 0, 30], 40, 48
    x, w, g = randn(1, 43, k), randn(2, 3, n, k), randn(3, 43, n)
    u, v = np64(randn(4, 43, k)), np64(randn(5, 3, n, k))
    ms = sizes(counts)

    def f(t):
        return sum((np64(g)[a:b] * ((np64(x) + t * u)[a:b] @ (np64(w)[e] + t * v[e]).T)).sum()
                   for e, (a, b) in enumerate(bounds(counts)))
    slope = (f(0.5) - f(-0.5))
    dx, dw = fx.grouped_mm(g, w, ms, transposed=True), fx.grouped_mm_weight_grad(g, x, ms)
    got = (np64(dx) * u).sum() + (np64(dw) * v).sum()
    # dx is rounded to bf16 (2^-8 relative), dw is fp32
    tol = 2.0 ** -8 * np.abs(np64(dx) * u).sum() + 2.0 ** -16 * np.abs(np64(dw) * v).sum()
    assert abs(got - slope) <= tol


def test_refusals():
    x, w, ms = randn(1, 8, 64), randn(2, 2, 32, 64), sizes([4, 4])
    dy = randn(3, 8, 32)
    bad = [
        (TypeError, lambda: fx.grouped_mm(x.float(), w.float(), ms)),
        (TypeError, lambda: fx.grouped_mm(x, w.half(), ms)),
        (TypeError, lambda: fx.grouped_mm(x, w, ms.int())),
        (TypeError, lambda: fx.grouped_mm(x, None, ms)),
        (TypeError, lambda: fx.grouped_mm(None, w, ms)),
        (ValueError, lambda: fx.grouped_mm(x, w, ms, transposed=True)),
        (ValueError, lambda: fx.grouped_mm(x, w[0], ms)),
        (ValueError, lambda: fx.grouped_mm(x, w, ms[:1])),
        (ValueError, lambda: fx.grouped_mm(x, w.transpose(1, 2), ms, transposed=True)),
        (ValueError, lambda: fx.grouped_mm(x.t(), w, ms)),
        (ValueError, lambda: fx.grouped_mm(x.cpu(), w, ms)),
        (ValueError, lambda: fx.grouped_mm(x, w.cpu(), ms)),
        (ValueError, lambda: fx.grouped_mm(x, w, ms, out=dy[:4])),
        (TypeError, lambda: fx.grouped_mm(x, w, ms, out=dy.float())),
        (ValueError, lambda: fx.grouped_mm(x.expand(8, 8, 64), w, ms)),
        (TypeError, lambda: fx.grouped_mm_weight_grad(dy, x.half(), ms)),
        (TypeError, lambda: fx.grouped_mm_weight_grad(dy.float(), x.float(), ms)),
        (TypeError, lambda: fx.grouped_mm_weight_grad(dy, x, ms, dtype=FP16)),
        (TypeError, lambda: fx.grouped_mm_weight_grad(dy, x, None)),
        (ValueError, lambda: fx.grouped_mm_weight_grad(dy[:7], x, ms)),
        (TypeError, lambda: fx.grouped_mm_weight_grad(dy, x, ms, dtype=BF16,
                                                      add=torch.zeros(2, 32, 64, device="cuda"))),
        (ValueError, lambda: fx.grouped_mm_weight_grad(
            dy, x, ms, add=torch.zeros(2, 64, 32, device="cuda"))),
        (ValueError, lambda: fx.grouped_mm_weight_grad(
            dy, x, ms, out=torch.zeros(3, 32, 64, device="cuda"))),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was taken")
