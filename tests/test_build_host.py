"""The build of the library and of the Python module beside it, with a stand-in for
nvcc that writes empty files."""
import os
import stat
import warnings

import pytest

from ragged_softmax_attention_gb300 import build as fwbuild


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build() into an empty folder."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do if [ "$1" = -o ]; then : > "$2"; fi; shift; done\n')
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(fwbuild, "_nvcc", lambda: str(nvcc))
    monkeypatch.setattr(fwbuild, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(fwbuild, "LIB", str(tmp_path / "libfw_attn.so"))
    monkeypatch.setattr(fwbuild, "fast_path", lambda: str(tmp_path / "_fw_fast.so"))
    return tmp_path


def raising(e):
    def f(out):
        raise e
    return f


@pytest.mark.parametrize("command", [
    lambda out: ["sh", "-c", "echo Python.h: No such file; exit 1"],
    lambda out: ["/no/such/compiler", out],
    raising(ModuleNotFoundError("No module named 'torch'")),
], ids=["headers", "compiler", "torch"])
def test_the_library_does_not_need_the_module(tree, monkeypatch, command):
    monkeypatch.setattr(fwbuild, "_fast_command", command)
    (tree / "_fw_fast.so").write_text("of older sources")
    os.utime(tree / "_fw_fast.so", (1, 1))
    with pytest.warns(RuntimeWarning, match="_fw_fast"):
        assert fwbuild.build() == str(tree / "libfw_attn.so")
    assert (tree / "libfw_attn.so").exists() and not (tree / "_fw_fast.so").exists()


def test_a_cuda_source_that_does_not_compile(tree, monkeypatch):
    monkeypatch.setattr(fwbuild, "_nvcc", lambda: "/bin/false")
    monkeypatch.setattr(fwbuild, "_fast_command", lambda out: ["touch", out])
    with pytest.raises(RuntimeError, match="nvcc failed"):
        fwbuild.build()
    assert not (tree / "libfw_attn.so").exists()


def test_an_up_to_date_module_stays(tree, monkeypatch):
    calls = []
    monkeypatch.setattr(fwbuild, "_fast_command", lambda out: calls.append(out) or ["touch", out])
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        fwbuild.build()
        fwbuild.build()
        assert len(calls) == 1
        fwbuild.build(force=True)
    assert len(calls) == 2


def test_a_module_of_other_versions_is_not_loaded(tree, monkeypatch):
    """Another torch makes a module of its own beside the first, and looks only there."""
    import torch

    from ragged_softmax_attention_gb300 import _binding
    monkeypatch.undo()
    monkeypatch.setattr(fwbuild, "HERE", str(tree))
    monkeypatch.setattr(fwbuild, "_nvcc", lambda: str(tree / "nvcc"))
    monkeypatch.setattr(fwbuild, "BUILD", str(tree / "_build"))
    monkeypatch.setattr(fwbuild, "LIB", str(tree / "libfw_attn.so"))
    monkeypatch.setattr(fwbuild, "_fast_command", lambda out: ["touch", out])
    fwbuild.build()
    first = fwbuild.fast_path()
    assert os.path.exists(first)
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert fwbuild.fast_path() != first
    monkeypatch.setattr(_binding, "_fast_module", None)
    with pytest.raises(RuntimeError, match="not built"):
        _binding._fast()
    fwbuild.build()
    assert os.path.exists(first) and os.path.exists(fwbuild.fast_path())
