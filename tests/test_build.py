"""What build() needs: the library is nvcc's alone and is linked whatever else
is installed; the binding of the bounded-cache calls also needs torch, the
Python headers and g++.  A small source stands in for csrc/.  CPU only."""
import ctypes
import importlib.util
import os
import shutil

import pytest

from paged_kv_cache_192_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cpp").write_text('extern "C" int one(void) { return 1; }\n')
    binding = tmp_path / "bounded_calls.cpp"
    binding.write_text('extern "C" int two(void) { return 2; }\n')
    for name, value in (("CSRC", csrc), ("BUILD", tmp_path / "_build"), ("PKG", tmp_path),
                        ("LIB", tmp_path / "libpa_gb300.so"), ("BINDING_SRC", binding),
                        ("BINDING", tmp_path / "_bounded_calls.so")):
        monkeypatch.setattr(b, name, str(value))
    return tmp_path


def linked(path):
    return ctypes.CDLL(path).one() == 1


def test_library_and_binding(tree):
    assert linked(b.build()) and os.path.exists(b.BINDING)


def test_without_torch_the_library_is_built(tree, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    assert linked(b.build())
    assert not os.path.exists(b.BINDING)
    assert linked(b.build())  # and again, from the cached objects


@pytest.mark.parametrize("cause", ["no g++", "no headers"])
def test_a_binding_that_fails_is_an_error_behind_the_library(tree, monkeypatch, cause):
    if cause == "no g++":
        which = shutil.which
        monkeypatch.setattr(shutil, "which",
                            lambda name, *a, **k: None if name in ("g++", "c++") else which(name, *a, **k))
    else:
        (tree / "bounded_calls.cpp").write_text("#include <no_such_header.h>\n")
    with pytest.raises(RuntimeError, match=r"g\+\+"):
        b.build()
    assert linked(b.LIB)
    assert not os.path.exists(b.BINDING)


def test_binding_built_once_torch_is_there(tree, monkeypatch):
    find = importlib.util.find_spec
    with monkeypatch.context() as m:
        m.setattr(importlib.util, "find_spec",
                  lambda name, *a: None if name == "torch" else find(name, *a))
        b.build()
    b.build()
    assert linked(b.LIB) and os.path.exists(b.BINDING)


def test_calls_without_the_binding_say_how_to_build_it(monkeypatch):
    from paged_kv_cache_192_gb300 import ops
    b.build()

    def missing(name, *a):
        raise ModuleNotFoundError(name)
    monkeypatch.setattr(ops, "_bounded", None)
    monkeypatch.setattr(importlib, "import_module", missing)
    with pytest.raises(RuntimeError, match="_bounded_calls.so is missing"):
        ops.compact_cache(None, None, None, None, None, None)
