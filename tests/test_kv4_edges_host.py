"""The 4-bit cache's host side without a GPU: the compiled binding's loading and building, and sizes at the ends."""

import os
import shutil
import subprocess

import pytest
import torch

import exact_io_aware_84_b200 as fa

HAVE_CC = shutil.which("gcc") is not None


class _CudaTensor(torch.Tensor):
    """Says of itself what _compiled asks."""

    is_cuda = True


@pytest.fixture
def fresh(monkeypatch):
    """_compiled as in a process that has not called it yet, for a tensor that passes for a CUDA one."""
    monkeypatch.setattr(fa, "_SERVE", None)
    t = torch.empty(0).as_subclass(_CudaTensor)
    monkeypatch.setattr(fa, "_torch", lambda: type("torch", (), {"Tensor": _CudaTensor}))
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
        pytest.skip("_serve.so not built")
    module = fa._compiled(fresh)
    assert module is not None and module is fa._compiled(fresh)
    assert all(callable(getattr(module, name)) for name in ("write", "read", "fwd"))
