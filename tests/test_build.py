"""What the in-tree build compiles, and what for: the library needs nvcc alone,
and only the binding's module depends on PyTorch.  CPU only."""

import ctypes
import os
import sys

import pytest

from paged_kv_cache_124_gb300 import build as b


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A source tree of one small translation unit, with outputs of its own."""
    csrc = tmp_path / "csrc"
    (csrc / "binding").mkdir(parents=True)
    (csrc / "one.cu").write_text('extern "C" int answer() { return 42; }\n__global__ void kernel() {}\n')
    binding = csrc / "binding" / "calls.cpp"
    binding.write_text("")
    monkeypatch.setattr(b, "CSRC", str(csrc))
    monkeypatch.setattr(b, "BINDING", str(binding))
    monkeypatch.setattr(b, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(b, "MODULE", str(tmp_path / "_one.so"))
    monkeypatch.setattr(b, "TORCH_STAMP", str(tmp_path / "obj" / "torch_version"))
    return tmp_path


def fail(*_):
    raise AssertionError("not to be built")


def test_the_library_needs_nvcc_alone(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)              # import torch raises
    monkeypatch.setattr(b, "_cxx", fail)
    assert b.build_library() == b.LIB and ctypes.CDLL(b.LIB).answer() == 42
    monkeypatch.setattr(b, "_compile", fail)
    assert b.build_library() == b.LIB                            # current: nothing to compile
    assert not os.path.exists(b.MODULE)


def test_a_module_that_cannot_be_built_leaves_the_library(tree, monkeypatch):
    def broken():
        raise RuntimeError("no PyTorch headers")
    monkeypatch.setattr(b, "_compile_binding", broken)
    with pytest.raises(RuntimeError, match="no PyTorch headers"):
        b.build()
    assert ctypes.CDLL(b.LIB).answer() == 42


def test_another_pytorch_builds_the_module_alone(tree, monkeypatch):
    import torch
    b.build_library()
    built = []

    def link(obj):
        built.append(obj)
        with open(b.LIB, "rb") as src, open(b.MODULE, "wb") as dst:
            dst.write(src.read())
        with open(b.TORCH_STAMP, "w") as f:
            f.write(torch.__version__)

    monkeypatch.setattr(b, "_compile", fail)
    monkeypatch.setattr(b, "_compile_binding", lambda: "object")
    monkeypatch.setattr(b, "_link_binding", link)
    b.build()
    b.build()                                                    # current
    assert built == ["object"]
    with open(b.TORCH_STAMP, "w") as f:
        f.write("0.0")
    b.build()
    assert built == ["object"] * 2


def test_a_newer_source_builds_what_it_belongs_to(tree, monkeypatch):
    import torch
    b.build_library()
    with open(b.LIB, "rb") as src, open(b.MODULE, "wb") as dst:
        dst.write(src.read())
    with open(b.TORCH_STAMP, "w") as f:
        f.write(torch.__version__)
    assert b.library_up_to_date() and b.module_up_to_date()
    later = os.path.getmtime(b.MODULE) + 10
    os.utime(b.BINDING, (later, later))
    assert b.library_up_to_date() and not b.module_up_to_date()
    os.utime(os.path.join(b.CSRC, "one.cu"), (later, later))
    assert not b.library_up_to_date()


def test_the_entry_points_can_be_run_as_a_script():
    """python __graft_entry__.py --smoke calls what the whole file defines."""
    import ast
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "__graft_entry__.py")
    with open(path) as f:
        body = ast.parse(f.read()).body
    main = [isinstance(n, ast.If) and "__name__" in ast.unparse(n.test) for n in body]
    assert main.count(True) == 1 and main[-1]
