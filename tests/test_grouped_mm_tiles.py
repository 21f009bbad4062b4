"""The 16-bit products on the GPU where a call is more than a round of tiles, or less: CTA pairs that
take many tiles of several stages, experts with more than eight row tiles, contractions in parts.
Every element is compared, in 64 bits on the GPU.

Tolerance: the tensor core's sums of 1024 terms (512 for fp32 gradients) take 64 (32) steps that lose
at most 2^-23 of what has been summed each; these sums, the parts of a contraction and what is added
are rounded once each, 2^-24; and the result, half of its type's eps.
"""
import pytest
import torch

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from test_grouped_mm import randn, shifted, sizes, strided, stream

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")
PARTS = 16


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


def check(got, want, magnitudes, terms, what):
    each = 512 if got.dtype == FP32 else 1024
    lost = min(terms, each) / 16 + 1
    tol = (lost * 2.0 ** -23 + (terms / each + PARTS + 2) * 2.0 ** -24) * magnitudes
    tol = tol + torch.finfo(got.dtype).eps / 2 * (want.abs() + tol) + torch.finfo(got.dtype).tiny
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at " \
        f"{bad.nonzero()[0].tolist()}"


def check_mm(out, x, w, counts, transposed, what="out"):
    at = 0
    for e, c in enumerate(counts):
        a, m = x[at:at + c].double(), w[e].double()
        m = m if transposed else m.t()
        check(out[at:at + c], a @ m, a.abs() @ m.abs(), x.shape[1], f"{what}, expert {e}")
        at += c


def check_grad(dw, dy, x, counts, add=None, what="dw"):
    at = 0
    for e, c in enumerate(counts):
        a, b = dy[at:at + c].double().t(), x[at:at + c].double()
        want, mag = a @ b, a.abs() @ b.abs()
        if add is not None:
            want, mag = want + add[e].double(), mag + add[e].double().abs()
        check(dw[e], want, mag, max(c, 1), f"{what}, expert {e}")
        at += c


def operands(counts, n, k, transposed, dtype, spare=0):
    m = sum(counts)
    x = torch.full((m + spare, k), NAN, dtype=dtype, device="cuda")
    x[:m] = randn(1, m, k, dtype=dtype)
    w = randn(2, len(counts), *((k, n) if transposed else (n, k)), dtype=dtype, scale=k ** -0.5)
    return x, w


UNEVEN = [257, 3, 511, 0, 130, 769, 1, 255] * 5


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,n,k", [([2600, 0, 4100, 33], 2056, 520), ([2600, 0, 4100, 33], 2056, 1160),
                                        (UNEVEN, 1032, 776), (UNEVEN, 1031, 777), (UNEVEN, 1029, 2100),
                                        (UNEVEN, 520, 3080), ([5000], 4104, 1032)])
def test_many_tiles(counts, n, k, transposed, dtype):
    """Several tiles per CTA pair, of different heights, and up to 20 row tiles of an expert."""
    x, w = operands(counts, n, k, transposed, dtype, spare=40)
    m = sum(counts)
    out = torch.full((m + 40, n), 7.0, dtype=dtype, device="cuda")
    fx.grouped_mm(x, w, sizes(counts), transposed=transposed, out=out)
    check_mm(out, x, w, counts, transposed)
    assert (out[m:] == 7.0).all()


@pytest.mark.parametrize("dtype,grad", [(BF16, FP32), (BF16, BF16), (FP16, FP16)])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("counts,n,k", [([300, 0, 1100, 77], 2600, 1032), ([40, 9, 0, 200] * 3, 2311, 1033),
                                        ([1500, 0, 700] * 3, 1288, 1032), ([2500, 8, 16, 3] * 8, 776, 520)])
def test_weight_grad_many_tiles(counts, n, k, add, dtype, grad):
    m = sum(counts)
    dy, x = randn(1, m, n, dtype=dtype), randn(2, m, k, dtype=dtype)
    before = randn(3, len(counts), n, k, dtype=grad) if add else None
    dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=before, dtype=grad)
    check_grad(dw, dy, x, counts, before)
    if add:     # in place: the same bits
        assert torch.equal(fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=before, out=before), dw)


def split_of(x, w, counts, n, k, transposed):
    """Parts of the contraction, from the workspace behind the operands' copies."""
    m, g = x.shape[0], len(counts)
    ld = x.stride(0)

    def copied(rows, cols, ld, at):
        if at % 16 == 0 and (ld % 8 == 0 or rows <= 1):
            return 0
        return -(-rows * (-(-cols // 8) * 8) * 2 // 256) * 256
    rows, cols = (g * k, n) if transposed else (g * n, k)
    copies = copied(rows, cols, cols, w.data_ptr()) + copied(m, k, ld, x.data_ptr())
    nbytes = fx.mslkb_grouped_mm_workspace_bytes(x.data_ptr(), w.data_ptr(), m, g, n, k, ld,
                                                 int(transposed))
    slices = (nbytes - copies) / (4 * -(-m * n // 4) * 4)
    assert slices == int(slices)
    return int(slices)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("n,k", [(72, 2048), (72, 4096), (72, 2001), (71, 4099), (333, 6000)])
@pytest.mark.parametrize("make", [lambda t: t, shifted, lambda t: strided(t, 5)])
def test_parts(make, n, k, transposed, dtype):
    """Few tiles, long contractions; operands that are copied first share the workspace."""
    counts, spare = [30, 0, 10], 9
    x, w = operands(counts, n, k, transposed, dtype, spare)
    x = make(x)
    assert split_of(x, w, counts, n, k, transposed) > 1
    m = sum(counts)
    for off in (False, True):
        out = torch.full((m + spare, n), 7.0, dtype=dtype, device="cuda")
        out = shifted(out) if off else out
        fx.grouped_mm(x, w, sizes(counts), transposed=transposed, out=out)
        check_mm(out, x, w, counts, transposed)
        assert (out[m:] == 7.0).all()


@pytest.mark.parametrize("transposed", [False, True])
def test_parts_of_clamped_counts(transposed):
    n, k = 72, 4096
    x, w = operands([30, 0, 10], n, k, transposed, BF16)
    assert split_of(x, w, [0] * 3, n, k, transposed) > 1
    for counts, real in (([30, -4, 1 << 40], [30, 0, 10]), ([1 << 62, 5, 5], [40, 0, 0])):
        out = fx.grouped_mm(x, w, sizes(counts), transposed=transposed)
        assert fx.device_status() == fx.MSLKB_DEV_MSIZES_CLAMPED
        check_mm(out, x, w, real, transposed)


@pytest.mark.parametrize("k", [4096, 2001])
def test_parts_on_streams_and_in_graphs(k):
    """Two calls at once, and two graphs replayed side by side with other counts: each with slices
    of its own."""
    n, counts = 72, [[30, 0, 10], [1, 35, 4]]
    data = [operands([40, 0, 0], n, k, t, BF16) for t in (False, True)]
    data = [(randn(9 + i, 40, k), w) for i, (_, w) in enumerate(data)]
    assert split_of(*data[0], [0] * 3, n, k, False) > 1
    ms = [sizes(c) for c in counts]
    outs = [torch.zeros((40, n), dtype=BF16, device="cuda") for _ in data]
    torch.cuda.synchronize()
    streams = [stream(), stream()]
    for _ in range(20):
        for (x, w), m, out, s, t in zip(data, ms, outs, streams, (False, True)):
            fx.grouped_mm(x, w, m, transposed=t, out=out, stream=s)
    torch.cuda.synchronize()
    for (x, w), c, out, t in zip(data, counts, outs, (False, True)):
        check_mm(out, x, w, c, t)
    graphs = []
    for (x, w), m, out, t in zip(data, ms, outs, (False, True)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fx.grouped_mm(x, w, m, transposed=t, out=out)
        graphs.append(graph)
    for m, c in zip(ms, reversed(counts)):
        m.copy_(sizes(c))
    for out in outs:
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (x, w), c, out, t in zip(data, reversed(counts), outs, (False, True)):
        check_mm(out, x, w, c, t)


def test_parts_do_not_change():
    x, w = operands([30, 0, 10], 72, 4096, False, BF16)
    ms = sizes([30, 0, 10])
    first = fx.grouped_mm(x, w, ms)
    assert all(torch.equal(fx.grouped_mm(x, w, ms), first) for _ in range(5))


@pytest.mark.parametrize("counts", [[9000], [5000, 40], [0, 3000, 1]])
@pytest.mark.parametrize("grad,dtype", [(FP32, BF16), (BF16, BF16), (FP16, FP16)])
def test_weight_grad_in_parts(counts, grad, dtype):
    """Rows in parts, whose ends lie inside an expert's rows or past them."""
    n, k = 64, 136
    m, g = sum(counts), len(counts)
    dy, x = randn(1, m, n, dtype=dtype), randn(2, m, k, dtype=dtype)
    nbytes = fx.mslkb_grouped_mm_weight_grad_workspace_bytes(dy.data_ptr(), x.data_ptr(), m, g, n, k,
                                                             n, k)
    assert nbytes >= 2 * 4 * g * n * k
    before = randn(3, g, n, k, dtype=grad)
    for add in (None, before):
        dw = fx.grouped_mm_weight_grad(dy, x, sizes(counts), add=add, dtype=grad)
        check_grad(dw, dy, x, counts, add)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("n,k", [(1000, 1160), (1001, 2100), (4104, 1032)])
def test_few_rows_of_many_experts(n, k, transposed, dtype):
    """Tiles narrower than others, and contractions longer than the tensor core's sums."""
    counts = [1, 3, 0, 2, 40] * 12
    x, w = operands(counts, n, k, transposed, dtype, spare=3)
    out = torch.full((sum(counts) + 3, n), 7.0, dtype=dtype, device="cuda")
    assert split_of(x, w, counts, n, k, transposed) == 0
    fx.grouped_mm(x, w, sizes(counts), transposed=transposed, out=out)
    check_mm(out, x, w, counts, transposed)
    assert (out[sum(counts):] == 7.0).all()
