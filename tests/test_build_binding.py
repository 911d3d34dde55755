"""build() makes the library whether or not the compiled binding can be built beside it."""
import os
import shutil
import warnings

import pytest

from paged_kv_cache_285_gb300 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A library of one small source and its binding, in a folder of their own."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "calls.cpp").write_text('extern "C" int one();\nextern "C" int two() { return 2 * one(); }\n')
    for name, at in (("HERE", tmp_path), ("CSRC", src), ("BUILD", tmp_path / "_build"), ("LIB", tmp_path / "libpkv.so"),
                     ("CALLS", tmp_path / "_calls.so"), ("CALLS_SRC", tmp_path / "calls.cpp")):
        monkeypatch.setattr(B, name, str(at))
    return tmp_path


def made(tree):
    return (tree / "libpkv.so").exists(), (tree / "_calls.so").exists()


def test_both_are_built_and_kept(tree):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        B.build()
        assert made(tree) == (True, True)
        at = [os.path.getmtime(tree / f) for f in ("libpkv.so", "_calls.so")]
        B.build()
    assert at == [os.path.getmtime(tree / f) for f in ("libpkv.so", "_calls.so")]


def test_a_binding_that_does_not_compile(tree):
    B.build()
    (tree / "calls.cpp").write_text("#include <no/such/header.h>\n")
    os.utime(tree / "calls.cpp", (2 ** 32, 2 ** 32))
    with pytest.warns(UserWarning, match="_calls.so was not built"):
        B.build()
    assert made(tree) == (True, False)      # the one there was is not kept beside another library
    (tree / "calls.cpp").write_text('extern "C" int two() { return 2; }\n')
    B.build()
    assert made(tree) == (True, True)


def test_no_host_compiler_for_the_binding(tree, monkeypatch):
    real = B._calls_cmd

    def missing():
        obj, cmd, lib = real()
        return obj, ["/no/such/g++"] + cmd[1:], lib
    monkeypatch.setattr(B, "_calls_cmd", missing)
    with pytest.warns(UserWarning, match="_calls.so was not built"):
        B.build()
    assert made(tree) == (True, False)


def test_no_torch_for_the_binding(tree, monkeypatch):
    def missing():
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(B, "_calls_cmd", missing)
    with pytest.warns(UserWarning, match="_calls.so was not built"):
        B.build()
    assert made(tree) == (True, False)


def test_a_binding_that_does_not_link(tree, monkeypatch):
    real = B._calls_cmd

    def elsewhere():
        obj, cmd, _ = real()
        return obj, cmd, str(tree / "nowhere")
    monkeypatch.setattr(B, "_calls_cmd", elsewhere)
    with pytest.warns(UserWarning, match="_calls.so was not built"):
        B.build()
    assert made(tree) == (True, False)


def test_a_library_that_does_not_compile_is_an_error(tree):
    (tree / "csrc" / "one.cu").write_text("#error no\n")
    with pytest.raises(RuntimeError):
        B.build()
    assert shutil.which("g++") and made(tree) == (False, False)
