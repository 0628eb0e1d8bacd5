"""The build of the library and of its Python binding, on sources of a line each."""
from __future__ import annotations

import os
import sys

import pytest

from chunked_gated_delta_02_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build's folders, moved to one with a kernel and a binding that compile in a second."""
    pkg = tmp_path / "pkg"
    csrc = pkg / "csrc"
    csrc.mkdir(parents=True)
    (csrc / "one.cu").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    (csrc / "binding.cpp").write_text('extern "C" int one(); int two() { return one() + 1; }\n')
    for name, path in (("PKG", pkg), ("CSRC", csrc), ("BUILD", pkg / "_build"), ("LIB", pkg / "libkda.so"),
                       ("BINDING", pkg / "_serving.so")):
        monkeypatch.setattr(build, name, str(path))
    return pkg


def test_library_and_binding(tree):
    assert build.build() == str(tree / "libkda.so")
    assert (tree / "_serving.so").exists()
    made = {f: os.stat(tree / f).st_mtime_ns for f in ("libkda.so", "_serving.so")}
    build.build()
    assert made == {f: os.stat(tree / f).st_mtime_ns for f in made}


def test_library_alone_without_torch(tree, monkeypatch):
    """The C interface needs no torch, and neither does its build."""
    monkeypatch.setitem(sys.modules, "torch", None)
    build.build()
    assert (tree / "libkda.so").exists() and not (tree / "_serving.so").exists()


def test_an_error_in_the_binding_leaves_the_library(tree):
    (tree / "csrc" / "binding.cpp").write_text("int two( { }\n")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert (tree / "libkda.so").exists()


def test_an_error_in_a_kernel_is_raised(tree):
    (tree / "csrc" / "one.cu").write_text("int one( { }\n")
    with pytest.raises(RuntimeError, match="one.cu"):
        build.build()
    assert not (tree / "libkda.so").exists()


def test_another_torch_builds_the_binding_anew(tree, tmp_path, monkeypatch):
    build.build()
    made = {f: os.stat(tree / f).st_mtime_ns for f in ("libkda.so", "_serving.so")}
    real, other = build._torch_dir(), tmp_path / "torch"
    other.mkdir()
    for name in ("include", "lib"):
        (other / name).symlink_to(os.path.join(real, name))
    (other / "version.py").write_text("__version__ = '0.0.1'\n")
    monkeypatch.setattr(build, "_torch_dir", lambda: str(other))
    build.build()
    after = {f: os.stat(tree / f).st_mtime_ns for f in made}
    assert after["libkda.so"] == made["libkda.so"] and after["_serving.so"] > made["_serving.so"]
    build.build()
    assert after == {f: os.stat(tree / f).st_mtime_ns for f in made}
