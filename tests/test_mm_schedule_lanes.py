"""The experts' rows of the 16-bit products, worked out on the CPU by the kernel's own source
(tests/lanes): counts that are to be clamped up to the largest number of rows that a call may have,
where 32 bits hold a sum of two counts no more."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from fp8_rowwise_scaled_gb300 import build as fxbuild

HERE = os.path.dirname(os.path.abspath(__file__))
MOST = 1 << 30
CLAMPED = 2


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    """grouped_mm.cuh's parameters and schedule, for the host compiler."""
    folder = tmp_path_factory.mktemp("lanes")
    with open(os.path.join(fxbuild.CSRC, "grouped_mm.cuh")) as f:
        source = f.read()

    def part(start, end):
        assert source.count(start) == 1 and source.count(end) == 1, (start, end)
        return source[source.index(start):source.index(end)]
    text = part("struct MmParams {", "// Tensor maps.  p, q: the operands") + \
        part("// Rows a and b together", "// kind::f16 MMA, fp32 accumulator")
    (folder / "schedule.cpp").write_text(
        '#include "lanes.h"\n'
        "inline int32_t __shfl_up_sync(uint32_t, int32_t v, int d) {\n"
        "  const int lane = lanes::g_cta->current->index % 32;\n"
        "  return static_cast<int32_t>(lanes::exchange(v)[lane < d ? lane : lane - d]);\n}\n"
        "inline int32_t __shfl_sync(uint32_t, int32_t v, int from) {\n"
        "  return static_cast<int32_t>(lanes::exchange(v)[from]);\n}\n"
        "inline bool __any_sync(uint32_t, bool v) {\n"
        "  const uint32_t* all = lanes::exchange(v);\n"
        "  return std::any_of(all, all + 32, [](uint32_t x) { return x != 0; });\n}\n"
        "inline void atomicOr(uint32_t* p, uint32_t v) { *p |= v; }\n"
        "namespace mslkb {\nconstexpr uint32_t kStatusClamped = 2u;\n" + text +
        '#include "mm_schedule.cpp"\n}  // namespace mslkb\n')
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(fxbuild.nvcc())))
    out = str(folder / "libschedule.so")
    r = subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-w", "-fwrapv", "-std=c++17", "-fPIC",
                        "-shared", "-I", os.path.join(HERE, "lanes"), "-isystem",
                        os.path.join(cuda, "include"), str(folder / "schedule.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return ctypes.CDLL(out)


def schedule(lib, counts, total, ct, grad, R=0):
    m = np.array(counts, dtype=np.int64)
    first, pre = np.full(len(m) + 1, -7, np.int32), np.full(len(m) + 1, -7, np.int32)
    tiles, status = np.zeros(1, np.int32), np.zeros(1, np.uint32)
    p = [a.ctypes.data_as(ctypes.c_void_p) for a in (m, first, pre, tiles, status)]
    assert lib.run_schedule(int(grad), p[0], len(m), total, ct, R, p[1], p[2], p[3], p[4]) == 0
    return first.tolist(), pre.tolist(), int(tiles[0]), int(status[0])


def expected(counts, total, ct):
    first, pre, clamped = [0], [0], False
    for m in counts:
        rows = min(max(m, 0), total - first[-1])
        clamped |= rows != m
        first.append(first[-1] + rows)
        pre.append(pre[-1] + ct * -(-rows // 256))
    return first, pre, CLAMPED if clamped else 0


def lists(total):
    yield [total]
    yield [total, total]
    yield [total - 1, 1, 0, 5]
    yield [total - 1, 2]
    yield [total // 2, total // 2 + 1, total]
    yield [-1, total, -(1 << 62), 1 << 62]
    yield [total] * 32
    yield [total] * 33
    yield [total // 40] * 40 + [total] * 60
    yield [total // 2 + 1] * 1024
    yield [0] * 1000 + [total] * 24
    yield [3, 0, 300] * 5


@pytest.mark.parametrize("total", [MOST, MOST - 1, MOST // 2 + 1, 1000, 1, 0])
def test_counts_are_clamped(lib, total):
    for counts in lists(total):
        want_first, want_pre, status = expected(counts, total, 1)
        first, pre, tiles, got = schedule(lib, counts, total, 1, False)
        assert first == want_first, counts[:4]
        assert pre == want_pre and tiles == want_pre[-1], counts[:4]
        assert got == status, counts[:4]
        first, _, tiles, got = schedule(lib, counts, total, 2, True, R=300)
        assert first == want_first and tiles == len(counts) * 2 * 2 and got == status, counts[:4]


def test_rows_together(lib):
    for a, b, total in ((MOST, MOST, MOST), (MOST - 1, 2, MOST), (0, 0, 0), (5, 6, 20), (5, 16, 20)):
        assert lib.run_add_rows(a, b, total) == min(total, a + b)
