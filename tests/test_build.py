"""The build: what counts as current, and the Python call module beside the library."""

import importlib.machinery
import os
import sys

import pytest

from int4_token_head_gb300 import _lib, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


needs_module = pytest.mark.skipif(build._binding_command() is None, reason="the call module cannot be built here")


def test_the_call_module_is_named_for_its_interpreter(monkeypatch):
    """Another interpreter on the same tree neither imports it nor finds its stamp current."""
    name = os.path.basename(build.BINDING_PATH)
    assert name[len("_fp8_binding"):] == importlib.machinery.EXTENSION_SUFFIXES[0]
    assert sys.implementation.cache_tag.replace("cpython-", "") in name
    before = build._fingerprint()
    monkeypatch.setattr(build, "PYTHON_TAG", ".cpython-399-somewhere.so")
    assert build._fingerprint() != before


@needs_module
def test_a_missing_call_module_is_built_again_alone(tmp_path, monkeypatch):
    assert build.is_current() and _lib._calls() is not _lib._Calls
    there = os.stat(build.LIB_PATH)
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / os.path.basename(build.BINDING_PATH)))
    assert not build.is_current()
    build.build()
    assert build.is_current() and os.path.exists(build.BINDING_PATH)
    assert os.stat(build.LIB_PATH) == there


@needs_module
def test_a_call_module_that_does_not_build_is_an_error(tmp_path, monkeypatch):
    bad = tmp_path / "bad.cpp"
    bad.write_text("#error nothing to build\n")
    monkeypatch.setattr(build, "BINDING_SRC", str(bad))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "module.so"))
    with pytest.raises(RuntimeError, match="nothing to build"):
        build.build()
    assert not build.is_current()


def test_without_a_compiler_the_library_alone_is_current(tmp_path, monkeypatch):
    """The calls go through ctypes then; nothing is built again and again."""
    monkeypatch.setattr(build, "_binding_command", lambda: None)
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "module.so"))
    assert build.is_current()
