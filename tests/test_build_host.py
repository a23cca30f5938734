"""build(): what it compiles, in which order, and what it does without torch or a C++ compiler (no compiler runs here)."""
import os
import subprocess
import sys
import types

import pytest

from block_diagonal_linear_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Targets in an empty folder; compilers that write their output's name into a list and the file."""
    ran = []

    def check_call(cmd, **_):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        with open(out, "wb") as f:
            f.write(b"".join(a.split("=", 1)[1].strip('"').encode() + b"\0" for a in cmd if a.startswith("-DMX4_NATIVE_KEY=")))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libmonarch.so"))
    monkeypatch.setattr(B, "NATIVE_LIB", str(tmp_path / "_mx4_native.so"))
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(subprocess, "check_call", check_call)
    return ran


def targets(ran):
    return [os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in ran]


def test_the_c_library_comes_first_and_nothing_is_built_twice(tree):
    assert B.build() == B.LIB
    assert targets(tree)[-2:] == ["libmonarch.so", "_mx4_native.so"] and all(t.endswith(".o") for t in targets(tree)[:-2])
    n = len(tree)
    B.build()
    assert len(tree) == n
    B.build(force=True)
    assert len(tree) == 2 * n


def test_without_torch_the_c_library_is_built_all_the_same(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)   # import torch raises ImportError
    with pytest.warns(UserWarning, match="_mx4_native.so was not built"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.NATIVE_LIB)


@pytest.mark.parametrize("fault", [FileNotFoundError("g++"), subprocess.CalledProcessError(1, "g++")])
def test_without_a_cpp_compiler_the_c_library_is_built_all_the_same(tree, monkeypatch, fault):
    ok = subprocess.check_call

    def check_call(cmd, **kw):
        if B.NATIVE_SOURCE in cmd:
            raise fault
        ok(cmd, **kw)
    monkeypatch.setattr(subprocess, "check_call", check_call)
    with open(B.NATIVE_LIB, "wb") as f:   # of older sources
        f.write(b"old")
    os.utime(B.NATIVE_LIB, (1, 1))
    with pytest.warns(UserWarning, match="_mx4_native.so was not built"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.NATIVE_LIB)


def test_another_torch_rebuilds_the_native_half(tree, monkeypatch):
    B.build()
    del tree[:]
    import torch
    other = types.SimpleNamespace(__file__=torch.__file__, __version__=torch.__version__ + ".1", compiled_with_cxx11_abi=torch.compiled_with_cxx11_abi)
    monkeypatch.setitem(sys.modules, "torch", other)
    B.build()
    assert targets(tree) == ["_mx4_native.so"]
    B.build()
    assert len(tree) == 1


def test_the_binding_refuses_a_native_half_of_another_torch(monkeypatch):
    import block_diagonal_linear_b200 as bdl
    bdl.Mx4
    from block_diagonal_linear_b200 import mx4
    assert mx4._native.key == B.native_key(mx4.torch)
    monkeypatch.setattr(mx4, "native_key", lambda t: "mx4 native: torch 0.0")
    with pytest.raises(RuntimeError, match="is built for .*torch 0.0"):
        mx4._load()
