"""The 4-bit cache's host side without a GPU: the compiled binding's loading and building, and sizes at the ends."""

import os
import shutil
import subprocess
import sys
import sysconfig

import pytest
import torch

import exact_io_aware_84_b200 as fa
from exact_io_aware_84_b200 import build
from test_binding_host import _FakeCuda

HAVE_CC = shutil.which("gcc") is not None


class _CudaTensor(torch.Tensor):
    """Says of itself what _compiled asks."""

    is_cuda = True


@pytest.fixture
def fresh(monkeypatch):
    """_compiled as in a process that has not called it yet, for a tensor that passes for a CUDA one."""
    monkeypatch.setattr(fa, "_SERVE", None)
    t = torch.empty(0).as_subclass(_CudaTensor)
    monkeypatch.setattr(fa, "_torch", lambda: type("torch", (), {"Tensor": _CudaTensor, "__version__": torch.__version__}))
    return t


@pytest.mark.parametrize("kind", ["not a library", pytest.param("unresolved", marks=pytest.mark.skipif(not HAVE_CC, reason="gcc not available"))])
def test_a_binding_that_does_not_load_leaves_the_other_way(kind, fresh, monkeypatch, tmp_path):
    path = tmp_path / "_serve.so"
    if kind == "unresolved":     # as after a change of the libraries that it was linked against
        src = tmp_path / "x.c"
        src.write_text("void no_such_symbol(void);\nvoid *PyInit__serve(void) { no_such_symbol(); return 0; }\n")
        subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(path)], check=True)
    else:
        path.write_bytes(b"\x7fELF and no more")
    monkeypatch.setattr(fa, "_serve_path", lambda: str(path))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert fa._compiled(fresh) is None
    path.unlink()
    assert fa._compiled(fresh) is None         # once is enough: no second try, no second warning


def test_no_binding_leaves_the_other_way(fresh, monkeypatch, tmp_path):
    monkeypatch.setattr(fa, "_serve_path", lambda: str(tmp_path / "none.so"))
    assert fa._compiled(fresh) is None


def test_the_binding_that_is_built_loads(fresh):
    if not os.path.exists(fa._serve_path()):
        pytest.skip("the binding is not built")
    module = fa._compiled(fresh)
    assert module is not None and module is fa._compiled(fresh)
    assert all(callable(getattr(module, name)) for name in ("write", "read", "fwd"))


def test_a_binding_of_another_python_or_torch_is_not_looked_at(monkeypatch):
    here = fa._serve_path()
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    other = fa._serve_path()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-299-x86_64-linux-gnu")
    assert len({here, other, fa._serve_path()}) == 3


@pytest.fixture
def compiler(monkeypatch, tmp_path):
    """Commands that the build of the binding runs, none of which is run; the binding lies in tmp_path."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc_path", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(fa, "_serve_path", lambda: str(tmp_path / "_serve.x.so"))
    return ran


def test_the_binding_is_built_when_it_is_old_or_asked_for(compiler, tmp_path):
    so = tmp_path / "_serve.x.so"
    build._build_serve()
    assert so.read_bytes() == b"built" and len(compiler) == 1
    build._build_serve()
    assert len(compiler) == 1
    build._build_serve(force=True)
    assert len(compiler) == 2
    os.utime(so, (1, 1))
    build._build_serve()
    assert len(compiler) == 3 and [p.name for p in tmp_path.iterdir()] == ["_serve.x.so"]


def test_a_forced_build_reaches_the_binding(monkeypatch):
    asked = []
    monkeypatch.setattr(build, "_compile", lambda *a: "")
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(cmd, 0, "", ""))
    monkeypatch.setattr(os, "replace", lambda a, b: None)
    monkeypatch.setattr(build, "_build_serve", lambda force=False: asked.append(force))
    build.build(force=True)
    assert asked == [True]


@pytest.mark.parametrize("missing", ["torch", "compiler", "headers"])
def test_the_library_is_built_where_the_binding_cannot_be(missing, compiler, monkeypatch, tmp_path):
    """What is there of older bindings goes, as the library that they were built for does."""
    monkeypatch.setattr(build, "_compile", lambda *a: "")
    so = tmp_path / "_serve.x.so"
    so.write_bytes(b"old")
    os.utime(so, (1, 1))
    lib = tmp_path / "libfa.so"
    monkeypatch.setattr(build, "LIB", str(lib))
    run = subprocess.run

    def no_binding(cmd, **kw):
        if cmd[0] != "g++":
            return run(cmd, **kw)
        if missing == "compiler":
            raise FileNotFoundError("g++")
        return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")

    monkeypatch.setattr(subprocess, "run", no_binding)
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(RuntimeWarning, match="not built"):
        assert build.build() == str(lib)
    assert lib.read_bytes() == b"built"
    assert not so.exists()


# ---------------------------------------------------------------- sizes at the ends


def test_no_pool_has_more_bytes_than_an_address_reaches():
    most = (1 << 31) - 1
    assert fa.fa_kv4_pool_bytes(most, 1, 16, 64) == most * 18 * 64
    assert fa.fa_kv4_pool_bytes(most, 1 << 16, 256, 128) == most * (1 << 16) * 16 * 18 * 128      # below 2^63
    for heads in (1 << 17, 1 << 18, 1 << 22, most):
        assert fa.fa_kv4_pool_bytes(most, heads, 256, 128) == 0
    with pytest.raises(ValueError):
        fa.fa_kv4_pool(most, 1 << 22, 256, 128, device="cpu")


def test_sizes_past_32_bits_are_not_cut():
    assert fa.fa_kv4_pool_bytes((1 << 32) + 1, 1, 16, 64) == 0
    assert fa.fa_kv4_pool_bytes(1, 1 << 32 | 1, 16, 64) == 0
    assert fa.fa_fwd_kv4_workspace_size((1 << 32) + 2, 8, 2, 1, 128) == 0
    assert fa.fa_fwd_kv4_workspace_size(2, 8, 2, (1 << 32) + 1, 128) == 0
    with pytest.raises(ValueError):
        fa.fa_kv4_pool((1 << 32) + 1, 1, 16, 64, device="cpu")


def test_a_table_past_32_bits_is_refused(monkeypatch):
    monkeypatch.setattr(fa, "load_library", lambda: pytest.fail("the library must not be reached"))
    rows = _FakeCuda((3, 4, 5, 64))
    cache = (_FakeCuda((7, 4, 2, 18 * 64), dtype=torch.uint8), _FakeCuda((3, (1 << 32) + 6), dtype=torch.int32),
             _FakeCuda((3,), dtype=torch.int32))
    for call in (lambda: fa.fa_kv4_write(rows, rows, *cache), lambda: fa.fa_fwd_kv4(rows, *cache),
                 lambda: fa.fa_kv4_read(*cache, k=rows, v=rows)):
        with pytest.raises(ValueError, match="2.31"):
            call()
