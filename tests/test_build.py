"""The build step on the host, with stand-ins for the compilers: the C library
does not depend on what the Python binding needs."""
import os
import stat
import subprocess

import pytest

from context_blockwise_causal_gb300 import _build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package directory, and a CUDA one whose nvcc writes its -o file."""
    pkg, nvcc = tmp_path / "pkg", tmp_path / "bin" / "nvcc"
    for d in (pkg, nvcc.parent, tmp_path / "include"):
        d.mkdir()
    (tmp_path / "include" / "cuda_runtime_api.h").touch()
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != "-o" ]; do shift; done\necho built > "$2"\n')
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(_build, "_nvcc", lambda: str(nvcc))
    monkeypatch.setattr(_build, "PKG_DIR", str(pkg))
    for name, path in (("LIB_PATH", "libcpattn.so"), ("CHECKED_LIB_PATH", "libcpattn_checked.so"),
                       ("BINDING_PATH", "_binding.so")):
        monkeypatch.setattr(_build, name, str(pkg / path))
    monkeypatch.setattr(_build, "_binding_command", lambda out: [str(nvcc), "-o", out])
    return pkg


def _built(tree):
    return {n for n in ("libcpattn.so", "libcpattn_checked.so", "_binding.so") if (tree / n).exists()}


def test_all_three_are_built(tree, monkeypatch):
    monkeypatch.setattr(_build, "_binding_lacks", lambda: None, raising=False)
    assert _build.build() == str(tree / "libcpattn.so")
    assert _built(tree) == {"libcpattn.so", "libcpattn_checked.so", "_binding.so"} and not _build.is_stale()


def test_the_library_is_built_where_the_binding_fails(tree, monkeypatch):
    (tree / "_binding.so").write_text("of another library")
    monkeypatch.setattr(_build, "_binding_lacks", lambda: None, raising=False)
    monkeypatch.setattr(_build, "_binding_command", lambda out: ["false"])
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()
    assert _built(tree) == {"libcpattn.so", "libcpattn_checked.so"} and _build.is_stale()


@pytest.mark.parametrize("missing", ["g++", "Python.h", "python_variable.h"])
def test_the_library_is_built_without_what_the_binding_needs(tree, monkeypatch, capfd, missing):
    (tree / "_binding.so").write_text("of another library")
    which, exists = _build.shutil.which, os.path.exists
    monkeypatch.setattr(_build.shutil, "which", lambda n: None if n == missing else which(n))
    monkeypatch.setattr(_build.os.path, "exists", lambda p: not str(p).endswith(missing) and exists(p))
    monkeypatch.setattr(_build, "_binding_command", lambda out: ["false"])
    assert _build.build() == str(tree / "libcpattn.so")
    assert _built(tree) == {"libcpattn.so", "libcpattn_checked.so"} and not _build.is_stale()
    assert missing in capfd.readouterr().err


def test_nothing_is_replaced_where_the_library_fails(tree, monkeypatch):
    for n in ("libcpattn.so", "libcpattn_checked.so", "_binding.so"):
        (tree / n).write_text("older")
    monkeypatch.setattr(_build, "_nvcc", lambda: "false")
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()
    assert all((tree / n).read_text() == "older" for n in ("libcpattn.so", "libcpattn_checked.so", "_binding.so"))


def test_this_machine_has_what_the_binding_needs():
    assert _build._binding_lacks() is None


def test_a_binding_for_another_pytorch_is_stale(tree, monkeypatch):
    """The binding uses PyTorch's C++ interface: under another version it is
    built again, and refused where it is not."""
    import torch

    monkeypatch.setattr(_build, "_binding_lacks", lambda: None)
    _build.build()
    _build.check_binding()
    assert not _build.is_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0")
        assert _build.is_stale()
        with pytest.raises(RuntimeError, match="2.0.0"):
            _build.check_binding()
        _build.build()
        _build.check_binding()
    with pytest.raises(RuntimeError, match="2.0.0"):
        _build.check_binding()
    os.remove(tree / "_binding.so")
    with pytest.raises(RuntimeError, match="missing"):
        _build.check_binding()
