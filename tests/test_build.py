"""What the build leaves where parts of its surroundings are missing (no GPU needed)."""
import ctypes
import os
import sysconfig
import types

import pytest
import torch

import causal_gqa_attention_rope_gb300 as na
from causal_gqa_attention_rope_gb300 import _build


@pytest.fixture
def outputs(monkeypatch, tmp_path):
    """The two outputs in a directory of their own (the library's objects stay where they are)."""
    _build.build()
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libna.so"))
    monkeypatch.setattr(_build, "CALLS", str(tmp_path / "_paged_calls.so"))
    return tmp_path


def check_library(path):
    lib = ctypes.CDLL(os.path.join(path, "libna.so"))
    lib.na_status_string.restype = ctypes.c_char_p
    assert lib.na_status_string(0) == b"ok"


@pytest.mark.parametrize("missing", ["torch", "torch_headers", "python_headers"])
def test_library_without_what_the_extension_module_needs(outputs, monkeypatch, missing):
    """libna.so is a plain C library: built and loaded without torch, its headers or Python.h."""
    empty = outputs / "empty"
    empty.mkdir()
    if missing == "python_headers":
        monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(empty)})
    else:
        spec = None if missing == "torch" else types.SimpleNamespace(
            submodule_search_locations=[str(empty)])
        monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: spec)
    with pytest.warns(UserWarning, match="paged calls"):
        assert _build.build() == str(outputs / "libna.so")
    assert sorted(p.name for p in outputs.iterdir()) == ["empty", "libna.so"]
    check_library(outputs)


def test_library_with_a_compiler_that_fails(outputs, monkeypatch):
    """An error while the extension module is compiled is raised, the library in place."""
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="paged_calls"):
        _build.build()
    check_library(outputs)


def test_another_torch_with_older_files(monkeypatch, tmp_path):
    """The module reads tensors through torch's inline code: with another torch installed it is
    compiled again, whatever the times of the files."""
    _build.build()
    real, other = os.path.dirname(torch.__file__), tmp_path / "torch"
    other.mkdir()
    for part in ("include", "lib"):
        (other / part).symlink_to(os.path.join(real, part))
    version = other / "version.py"
    version.write_text("__version__ = '1.0.0'\ngit_version = 'another'\n")
    os.utime(version, (1e9, 1e9))
    calls = types.SimpleNamespace(submodule_search_locations=[str(other)])
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: calls)
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="paged_calls"):  # it tries to
        _build.build()


def test_module_of_another_torch_is_refused(monkeypatch):
    _build.build()
    monkeypatch.setattr(na, "_native", None)
    monkeypatch.setattr(torch.version, "git_version", "another")
    with pytest.raises(RuntimeError, match="another torch"):
        na._calls()


def test_module_is_named_for_its_python():
    assert os.path.basename(_build.CALLS) == "_paged_calls" + sysconfig.get_config_var("EXT_SUFFIX")
