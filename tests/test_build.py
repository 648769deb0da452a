"""What the build makes of what is there, with the compilers replaced: the C library is linked whatever becomes of the
calls on PyTorch tensors, and each of the two is made again when something that went into it has changed."""
import os
import subprocess
import types

import pytest
import torch

from reduce_residual_rmsnorm_gb300 import build as libbuild


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty package folder; ``runs`` lists the compilers' calls, ``fails(command)`` chooses those that fail."""
    t = types.SimpleNamespace(runs=[], fails=lambda cmd: False, lib=str(tmp_path / "lib.so"), calls=str(tmp_path / "calls.so"))
    monkeypatch.setattr(libbuild, "LIB_PATH", t.lib)
    monkeypatch.setattr(libbuild, "CALLS_PATH", t.calls)
    monkeypatch.setattr(libbuild, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(libbuild, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")

    def run(cmd, **kw):
        t.runs.append(cmd)
        if t.fails(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(libbuild.subprocess, "run", run)
    return t


def _of_calls(cmd):
    return cmd[0] == "g++"


def test_both_are_built_once(tree):
    assert libbuild.build() == tree.lib
    assert os.path.exists(tree.lib) and os.path.exists(tree.calls)
    n = len(tree.runs)
    assert n == len(libbuild.sources()) + 3
    libbuild.build()
    assert len(tree.runs) == n


@pytest.mark.parametrize("step", ("-c", "-shared"))
def test_library_is_linked_where_the_calls_do_not_compile(tree, step):
    tree.fails = lambda cmd: _of_calls(cmd) and step in cmd
    with pytest.raises(RuntimeError, match="no such header"):
        libbuild.build()
    assert os.path.exists(tree.lib) and not os.path.exists(tree.calls)


def test_library_needs_no_cuda_in_pytorch(tree, monkeypatch):
    monkeypatch.setattr(torch.version, "cuda", None)
    assert libbuild.build() == tree.lib
    assert os.path.exists(tree.lib) and not any(_of_calls(c) for c in tree.runs)
    n = len(tree.runs)
    libbuild.build()
    assert len(tree.runs) == n
    monkeypatch.undo()


@pytest.mark.parametrize("before", (False, True), ids=("never", "uninstalled"))
def test_library_needs_no_pytorch(tree, monkeypatch, before):
    import builtins

    if before:  # the calls of an earlier build are there
        libbuild.build()
        tree.runs.clear()

    real = builtins.__import__

    def no_torch(name, *args, **kw):
        if name == "torch" or name.startswith("torch."):
            raise ImportError(name)
        return real(name, *args, **kw)

    monkeypatch.setattr(builtins, "__import__", no_torch)
    assert libbuild.up_to_date() == before
    assert libbuild.build() == tree.lib
    assert os.path.exists(tree.lib) and not any(_of_calls(c) for c in tree.runs)


def test_each_is_made_again_alone(tree):
    libbuild.build()
    for gone, n in ((tree.calls, 2), (tree.lib, len(libbuild.sources()) + 1)):
        os.remove(gone)
        tree.runs.clear()
        libbuild.build()
        assert os.path.exists(gone) and len(tree.runs) == n


@pytest.mark.parametrize("other", ("pytorch", "python"))
def test_calls_are_made_again_for_another_pytorch_or_python(tree, monkeypatch, other):
    libbuild.build()
    assert libbuild.calls_match()
    tree.runs.clear()
    if other == "pytorch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    else:
        real = libbuild.sysconfig.get_config_var
        monkeypatch.setattr(libbuild.sysconfig, "get_config_var", lambda n: "cpython-0" if n == "SOABI" else real(n))
    assert not libbuild.calls_match() and not libbuild.up_to_date()
    libbuild.build()
    assert [_of_calls(c) for c in tree.runs] == [True, True]
    assert libbuild.calls_match() and libbuild.up_to_date()


def test_calls_of_another_pytorch_are_not_loaded(monkeypatch):
    from reduce_residual_rmsnorm_gb300 import _nvfp4_moe

    libbuild.build()
    monkeypatch.setattr(_nvfp4_moe, "_calls", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="another PyTorch"):
        _nvfp4_moe._native()
    monkeypatch.undo()
    assert _nvfp4_moe._native() is not None


def test_calls_without_a_stamp_are_made_again(tree):
    libbuild.build()
    os.remove(os.path.join(libbuild.BUILD_DIR, libbuild.CALLS_STAMP))
    assert not libbuild.up_to_date()
    libbuild.build()
    assert libbuild.up_to_date()
