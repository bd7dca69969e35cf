"""The build's two steps, with compilers that only write their output file: the library needs no
torch, the native module belongs to one interpreter and one torch."""
import os
import stat
import sys

import pytest

from adapter_gemv_sgmv_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs under tmp_path; `nvcc` writes what -o names."""
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.parent.mkdir()
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho made > "$2"\n')
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setenv("CXX", str(nvcc))
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "liblora_sgmv.so"))
    return tmp_path


def _made(tree):
    return sorted(f for f in os.listdir(tree) if f.endswith(".so"))


def test_library_is_built_without_torch(tree, monkeypatch):
    for name in [m for m in sys.modules if m == "torch" or m.startswith("torch.")]:
        monkeypatch.setitem(sys.modules, name, None)         # (an import of it fails)
    monkeypatch.setitem(sys.modules, "torch", None)
    assert B.build(force=True) == B.LIB
    assert _made(tree) == ["liblora_sgmv.so"]


def test_library_is_built_with_a_torch_without_cuda(tree, monkeypatch):
    import torch
    monkeypatch.setattr(torch.version, "cuda", None)
    assert B.build(force=True) == B.LIB
    assert _made(tree) == ["liblora_sgmv.so"]


def test_library_stays_where_the_module_fails(tree, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(Exception):
        B.build(force=True)
    assert _made(tree) == ["liblora_sgmv.so"]


def test_module_of_another_torch_is_not_taken(tree, monkeypatch):
    import torch
    B.build(force=True)
    first = B.native_path()
    assert _made(tree) == sorted([os.path.basename(first), "liblora_sgmv.so"])
    made = os.stat(first).st_mtime_ns
    B.build()
    assert os.stat(first).st_mtime_ns == made               # up to date: left alone
    monkeypatch.setattr(torch, "__version__", "99.0.0+cu999")
    assert B.native_path() != first and not os.path.exists(B.native_path())
    B.build()
    assert len(_made(tree)) == 3
