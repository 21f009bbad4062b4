"""The norm's ring kernels on the CPU with their threads in chosen orders (tests/lanes): no lane
may depend on the others being as far as itself, and no copy on arriving early or late.  The
kernels' source is compiled as it stands; only barriers, shuffles, copies and the instructions
without a C++ form are replaced."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import moe_reference as ref
from fp8_rowwise_scaled_gb300 import build as fxbuild
from moe_reference import U, close, np64, rounding

HERE = os.path.dirname(os.path.abspath(__file__))
CODES = {torch.bfloat16: 0, torch.float32: 2}
REPLACED = ["max_nan", "recip", "pack_e4m3x4", "unpack_e4m3x2", "load32", "store32"]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """norm_quant.cu up to its launches, for the host compiler."""
    folder = tmp_path_factory.mktemp("lanes")
    with open(os.path.join(fxbuild.CSRC, "rows.cuh")) as f:
        rows = f.read()
    for name in REPLACED:   # those written in instructions of the device
        rows, n = re.subn(r"__device__ __forceinline__ [\w ]+ " + name + r"\([^{]*\) \{\n.*?\n\}\n",
                          "", rows, flags=re.S)
        assert n >= 1, name
    rows = rows.replace("struct Words8 {\n  uint32_t w[8];\n};", "struct Words8 {\n  uint32_t w[8];\n};\n"
                        "inline Words8 load32(const void* p) {\n  Words8 r;\n"
                        "  std::memcpy(&r, p, 32);\n  return r;\n}\n"
                        "inline void store32(void* p, const Words8& r) { std::memcpy(p, &r, 32); }")
    rows = re.sub(r"// e4m3 codes of columns that are all in the row\.\n.*?\n\}\n\n(?=\}  // namespace)", "",
                  rows, flags=re.S)
    with open(os.path.join(fxbuild.CSRC, "norm_quant.cu")) as f:
        source = f.read()
    assert source.count("// launches\n") == 1
    source = source.split("// launches\n")[0]
    source, n = re.subn(r"extern __shared__ __align__\(16\) uint8_t ring\[\];",
                        "uint8_t* const ring = lanes::g_ring;", source)
    assert n == 2
    (folder / "rows.cuh").write_text(rows)
    (folder / "ptx.cuh").write_text('#include "lanes.h"\n')
    (folder / "host.h").write_text('#include "lanes.h"\n')
    (folder / "norm.cpp").write_text('#include "lanes.h"\n' + source + "\n}  // namespace\n"
                                     '#include "norm_rings.cpp"\n}  // namespace mslkb\n')
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(fxbuild.nvcc())))
    out = str(folder / "libnorm.so")
    r = subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-w", "-std=c++17", "-fPIC", "-shared",
                        "-I", str(folder), "-I", os.path.join(HERE, "lanes"), "-isystem",
                        os.path.join(cuda, "include"), str(folder / "norm.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    L = ctypes.CDLL(out)
    p, i, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.run_norm_backward.argtypes = [i] * 4 + [p] * 7 + [i64] + [i] * 6
    L.run_norm_forward.argtypes = [i] * 3 + [p] * 8 + [i64] + [i] * 5
    return L


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g).to(dtype)


def address(t):
    return None if t is None else t.data_ptr()


FP32, BF16 = torch.float32, torch.bfloat16
SCHEDULES = [(order, late) for order in (0, 1, 2) for late in (0, 1)]


@pytest.mark.parametrize("order,late", SCHEDULES)
@pytest.mark.parametrize("dtype,vecs,stages,rows,H,x,y,T", [
    # 32-bit rows: lanes read pieces that others copied; the last warp's partly past the row's end
    (FP32, 1, 2, 1, 136, 32, 4, 40), (FP32, 1, 2, 1, 520, 96, 2, 13), (FP32, 1, 2, 0, 2056, 288, 1, 7),
    (FP32, 1, 2, 0, 256, 32, 1, 9), (FP32, 4, 2, 0, 1032, 64, 1, 9), (FP32, 4, 2, 0, 5128, 192, 1, 7),
    # 16-bit rows: each its own
    (BF16, 1, 2, 1, 136, 32, 4, 40), (BF16, 2, 3, 1, 264, 32, 3, 29), (BF16, 4, 2, 1, 520, 32, 4, 30),
    (BF16, 4, 2, 1, 1040, 64, 4, 21), (BF16, 2, 3, 0, 2056, 160, 1, 9), (BF16, 2, 2, 0, 1048, 96, 1, 9)])
def test_gradient(kernels, dtype, vecs, stages, rows, H, x, y, T, order, late):
    g = torch.Generator().manual_seed(H + T)
    dy, h, dres = (randn(g, T, H, dtype=dtype) for _ in range(3))
    w = randn(g, H, dtype=dtype)
    rstd = h.double().square().mean(-1).add(1e-6).rsqrt().float()
    grid = 2
    for residual in (dres, None):
        dx, parts = torch.zeros_like(dy), torch.full((grid, H), float("nan"))
        assert kernels.run_norm_backward(
            CODES[dtype], vecs, stages, rows, *map(address, (dy, h, w, rstd, residual, dx, parts)),
            T, H, grid, x, y, order, late) == 0
        a = [np64(t) for t in (dy, h, w, rstd)]
        want_dx, want_dw = ref.norm_backward(*a, None if residual is None else np64(residual))
        xhat, gg = a[1] * a[3][:, None], a[0] * a[2]
        size = a[3][:, None] * (np.abs(gg) + np.abs(xhat) * np.abs(gg * xhat).mean(-1, keepdims=True))
        # as on the device: 42 u of the mean's terms and the other terms' roundings
        close(dx, want_dx, rounding(dtype, want_dx) + 48 * U * size + 2 * U * np.abs(want_dx), "dx")
        # 20 rows of a thread, 4 rows side by side, 2 parts
        close(parts.double().sum(0), want_dw, 32 * U * np.abs(a[0] * xhat).sum(0), "dweight")


@pytest.mark.parametrize("order,late", SCHEDULES)
@pytest.mark.parametrize("dtype,vecs,stages,H,threads,residual,T", [
    (BF16, 1, 2, 1024, 64, True, 9), (BF16, 1, 3, 528, 64, False, 11), (BF16, 2, 2, 2064, 96, True, 7),
    (FP32, 1, 2, 528, 64, True, 9), (FP32, 1, 2, 384, 32, False, 9)])
def test_forward(kernels, dtype, vecs, stages, H, threads, residual, T, order, late):
    g = torch.Generator().manual_seed(H + T)
    x, res, w = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype), randn(g, H, dtype=dtype)
    want_h, want_rstd, want_y = ref.norm(np64(x), np64(res) if residual else None, np64(w), 1e-6)
    for blocks in ((0, 1) if H % 128 == 0 else (0,)):
        q = torch.zeros((T, H), dtype=torch.uint8)
        scale = torch.zeros((T, H // 128) if blocks else (T,))
        ro, y, rstd = torch.zeros_like(x), torch.zeros_like(x), torch.zeros(T)
        assert kernels.run_norm_forward(
            CODES[dtype], vecs, stages, *map(address, (x, res if residual else None, w, q, scale,
                                                       ro if residual else None, y, rstd)),
            T, H, blocks, 2, threads, order, late) == 0
        rel = 32 * U   # as on the device: half of the 42 u of the sum, and the roundings
        ref.check_codes(q, scale, want_y, ref.BLOCK if blocks else H, rel, "q")
        close(y, want_y, rounding(dtype, want_y) + rel * np.abs(want_y), "y")
        close(rstd, want_rstd, rel * want_rstd, "rstd")
        if residual:
            close(ro, want_h, rounding(dtype, want_h) + 2 * U * np.abs(want_h), "residual")
