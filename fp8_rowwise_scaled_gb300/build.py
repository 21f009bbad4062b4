"""Build libmslkb.so in-tree with nvcc for sm_103a (GB300).

    python -m fp8_rowwise_scaled_gb300.build [--force] [--ptxas-verbose] [--checked]

--checked builds libmslkb_checked.so instead: the same sources compiled with MSLKB_CHECKED,
whose kernels test every global access against the extents of the call's buffers and
report an index outside them in the device status word (MSLKB_DEV_BOUNDS) instead of
making the access.  A test build (the stand-in for a memory checker); slower.

Each translation unit in csrc/ compiles in parallel to _build/*.o, then nvcc links them
into fp8_rowwise_scaled_gb300/libmslkb.so (CUDA runtime linked statically; the CUDA driver's
tensor-map encoder is fetched at run time, so the library loads on a machine without a
GPU).  Rebuilds only when a source or header is newer than the library.  Beside it the host
compiler makes _binding.so, through which the torch forms of the operators around the
product reach the library (left out where torch with CUDA is not installed: the C library does
without).  It is also rebuilt when Python or torch is another than the one that it was compiled
against (_binding.so.against).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmslkb.so")
BUILD_CHECKED = os.path.join(PKG, "_build_checked")
LIB_CHECKED = os.path.join(PKG, "libmslkb_checked.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["mslkb.cu", "mslkb_noalloc.cu", "variants_stacked_tma.cu",
           "variants_dynamic_tma.cu", "variants_cpasync.cu", "variants_ragged_n.cu",
           "variants_ragged_k.cu", "variants_blockscale.cu", "variants_blockscale_dynamic.cu",
           "norm_quant.cu", "route.cu", "dispatch.cu", "swiglu_quant.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA 13 toolkit required to build libmslkb.so)")


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES] + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))
            + [os.path.abspath(__file__)])


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _compile(src: str, ptxas_verbose: bool, checked: bool = False) -> tuple[str, str]:
    obj = os.path.join(BUILD_CHECKED if checked else BUILD,
                       os.path.splitext(os.path.basename(src))[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
           "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if checked:
        cmd.insert(1, "-DMSLKB_CHECKED")
    if ptxas_verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False,
          checked: bool = False) -> str:
    """Compile and link libmslkb.so (checked: libmslkb_checked.so); returns its path."""
    lib = LIB_CHECKED if checked else LIB
    if not force and not ptxas_verbose and up_to_date(lib):
        if not checked:
            build_binding()
        return lib
    os.makedirs(BUILD_CHECKED if checked else BUILD, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        results = list(ex.map(lambda s: _compile(s, ptxas_verbose, checked), srcs))
    if verbose or ptxas_verbose:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if not checked:
        build_binding(force)
    return lib


def torch_folder():
    """(the folder of the installed torch, None), or (None, why the extension cannot be built)."""
    spec = importlib.util.find_spec("torch")   # found, not imported: seconds
    if spec is None:
        return None, "torch is not installed"
    folder = os.path.dirname(spec.origin)
    if not os.path.exists(os.path.join(folder, "lib", "libc10_cuda.so")):
        return None, f"torch in {folder} was built without CUDA"
    return folder, None


def _read(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def built_against(torch_dir: str) -> str:
    """The Python and the torch that an extension compiled now belongs to."""
    return f"{sys.version}\n{torch_dir}\n{_read(os.path.join(torch_dir, 'version.py'))}"


def build_binding(force: bool = False) -> str | None:
    """Compile _binding.so, the extension that checks torch tensors and passes them to
    libmslkb.so, with the host compiler against this Python and torch; returns its path.  Without
    torch (or with one that has no CUDA) there is nothing that it could serve: says so and
    returns None."""
    torch_dir, missing = torch_folder()
    if torch_dir is None:
        print(f"{os.path.basename(BINDING)} left out ({missing}); libmslkb.so does not need it",
              file=sys.stderr)
        return None
    inputs = [BINDING_SOURCE, os.path.join(INCLUDE, "mslkb.h"), os.path.abspath(__file__)]
    against = built_against(torch_dir)
    if not force and os.path.exists(BINDING) and _read(BINDING + ".against") == against and \
            all(os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in inputs):
        return BINDING
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), BINDING_SOURCE, "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
           "-lc10", "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {BINDING_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING + ".against", "w") as f:
        f.write(against)
    return BINDING


def load_binding():
    """The loaded extension (raises if it has not been built)."""
    if not os.path.exists(BINDING):
        missing = torch_folder()[1]
        raise RuntimeError(f"{BINDING} is missing: " + (
            f"{missing}, and the torch forms need torch with CUDA" if missing else
            "build it with `python -m fp8_rowwise_scaled_gb300.build`"))
    name = __package__ + "._binding"
    if name in sys.modules:
        return sys.modules[name]
    loader = importlib.machinery.ExtensionFileLoader(name, BINDING)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader(name, loader))
    loader.exec_module(module)
    sys.modules[name] = module
    return module


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    ap.add_argument("--checked", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=True, ptxas_verbose=a.ptxas_verbose, checked=a.checked))
