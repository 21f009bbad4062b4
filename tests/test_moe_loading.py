"""First use of the torch forms from several host threads, and the build of the extension behind
them, on the CPU."""
import os
import sys
import threading
import time
import types

import pytest

import fp8_rowwise_scaled_gb300 as fx
from fp8_rowwise_scaled_gb300 import build as fxbuild
from fp8_rowwise_scaled_gb300 import moe


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fxbuild.build()
    fx.lib()


@pytest.fixture
def unloaded(monkeypatch):
    """As before the first call (what is loaded now comes back afterwards)."""
    monkeypatch.setattr(moe, "_b", None)
    monkeypatch.setattr(moe, "_torch", None)


def in_threads(n, call):
    """Runs call(i) in n threads that start together; the exceptions that they raised."""
    errors, gate = [], threading.Barrier(n)

    def body(i):
        gate.wait()
        try:
            call(i)
        except BaseException as e:   # handed to the test
            errors.append(e)
    threads = [threading.Thread(target=body, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


def test_torch_is_there_before_the_extension(unloaded):
    """The callers look at the extension's name: at no line is it set and torch is not."""
    seen = []

    def trace(frame, event, arg):
        if frame.f_code.co_filename != moe.__file__:
            return None
        seen.append((moe._b is not None, moe._torch is not None))
        return trace

    sys.settrace(trace)
    try:
        moe._setup()
    finally:
        sys.settrace(None)
    assert seen and moe._b is not None and moe._torch is not None
    assert (True, False) not in seen


def test_first_calls_of_several_threads(unloaded, monkeypatch):
    """One load for all of them, and each call gets as far as its checks."""
    loads, load = [], fxbuild.load_binding

    def slow():
        loads.append(1)
        time.sleep(0.05)
        return load()
    monkeypatch.setattr(fxbuild, "load_binding", slow)

    def first(i):
        with pytest.raises(TypeError):
            fx.moe_combine([i], None)
    assert in_threads(8, first) == []
    assert len(loads) == 1



# ---------------------------------------------------------------------------------------
# the build where torch is missing or has changed
# ---------------------------------------------------------------------------------------
@pytest.fixture
def build_elsewhere(monkeypatch, tmp_path):
    """build() of the extension into an empty folder, with what it runs recorded: the compiler
    here writes an empty file."""
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(fxbuild, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(fxbuild, "subprocess", types.SimpleNamespace(run=run))
    return runs


@pytest.mark.parametrize("torch_is", ["missing", "without CUDA"])
def test_build_without_torch(build_elsewhere, monkeypatch, tmp_path, capsys, torch_is):
    """The C library needs neither torch nor the extension: build() says that it leaves the
    extension out, and a call of the torch forms says why it is not there."""
    folder = tmp_path / "torch"
    folder.mkdir()
    (folder / "__init__.py").write_text("")
    (folder / "version.py").write_text("__version__ = '2.9.1+cpu'\n")
    spec = types.SimpleNamespace(origin=str(folder / "__init__.py"))
    monkeypatch.setattr(fxbuild.importlib.util, "find_spec",
                        lambda name: None if torch_is == "missing" else spec)
    assert fxbuild.build() == fxbuild.LIB
    assert build_elsewhere == [] and not os.path.exists(fxbuild.BINDING)
    said = capsys.readouterr()
    assert "torch" in said.err + said.out
    monkeypatch.delitem(sys.modules, fxbuild.__package__ + "._binding", raising=False)
    with pytest.raises(RuntimeError, match="torch"):
        fxbuild.load_binding()


def test_build_again_for_another_torch_or_python(build_elsewhere, monkeypatch, tmp_path):
    """The extension belongs to the torch and the Python that it was compiled against."""
    fxbuild.build()
    fxbuild.build()
    assert len(build_elsewhere) == 1
    folder = tmp_path / "torch"
    (folder / "lib").mkdir(parents=True)
    (folder / "lib" / "libc10_cuda.so").write_text("")
    (folder / "__init__.py").write_text("")
    (folder / "version.py").write_text("__version__ = '2.9.1+cu130'\n")
    spec = types.SimpleNamespace(origin=str(folder / "__init__.py"))
    monkeypatch.setattr(fxbuild.importlib.util, "find_spec", lambda name: spec)
    fxbuild.build()
    fxbuild.build()
    assert len(build_elsewhere) == 2
    (folder / "version.py").write_text("__version__ = '2.11.0+cu130'\n")
    fxbuild.build()
    fxbuild.build()
    assert len(build_elsewhere) == 3
    monkeypatch.setattr(sys, "version", "3.14.0 (another)")
    fxbuild.build()
    fxbuild.build()
    assert len(build_elsewhere) == 4
