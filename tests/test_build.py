"""The build step's host logic (no compiler runs here)."""
import os
import subprocess
import sys
import types
import warnings

import pytest

import block_sparse_attention_selected_b200 as nsa
from block_sparse_attention_selected_b200 import build as nsa_build
from block_sparse_attention_selected_b200 import paged as npaged


@pytest.fixture
def bind_files(tmp_path, monkeypatch):
    """_paged_bind.so and its stamp in a folder of their own; the compiler calls are recorded."""
    monkeypatch.setattr(nsa_build, "LIB_BIND", str(tmp_path / "_paged_bind.so"))
    monkeypatch.setattr(nsa_build, "BIND_STAMP", str(tmp_path / "_build" / "paged_bind.txt"))
    calls = []

    def compile_(cmd):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(subprocess, "check_call", compile_)
    return calls


def test_the_library_is_built_without_the_module(monkeypatch):
    order = []
    monkeypatch.setattr(nsa_build, "_stale", lambda lib: True)
    monkeypatch.setattr(nsa_build, "_build_library", lambda lib, verbose, checks: order.append(lib))
    for problem in (FileNotFoundError("g++"), subprocess.CalledProcessError(1, "g++"), ImportError("torch")):
        def fail(force=False):
            order.append("bind")
            raise problem
        monkeypatch.setattr(nsa_build, "build_bind", fail)
        with pytest.warns(UserWarning, match="_paged_bind.so was not built"):
            assert nsa_build.build() == nsa_build.LIB
    assert order == [nsa_build.LIB, "bind"] * 3


def test_the_module_is_built_again_for_another_torch(bind_files, monkeypatch):
    nsa_build.build_bind()
    nsa_build.build_bind()
    assert len(bind_files) == 1
    monkeypatch.setattr(nsa_build, "bind_target", lambda: "cpython-399 torch 9.9")
    nsa_build.build_bind()
    nsa_build.build_bind()
    assert len(bind_files) == 2
    assert '-DNSA_BUILT_FOR="cpython-399 torch 9.9"' in bind_files[1]
    os.remove(nsa_build.LIB_BIND)
    nsa_build.build_bind()
    assert len(bind_files) == 3


def test_a_module_of_another_torch_is_not_used(monkeypatch):
    nsa_build.build()
    other = types.SimpleNamespace(built_for="cpython-399 torch 9.9", init=None)
    monkeypatch.setitem(sys.modules, "block_sparse_attention_selected_b200._paged_bind", other)
    monkeypatch.setattr(nsa, "_paged_bind", other, raising=False)
    monkeypatch.setattr(npaged, "_bind", None)
    with pytest.warns(UserWarning, match="built for cpython-399"):
        assert npaged._plain(None) is False
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert npaged._plain(None) is False      # said once


def test_the_module_that_was_built_is_used(monkeypatch):
    nsa_build.build()
    monkeypatch.setattr(npaged, "_bind", None)
    assert npaged._plain(None) is False and npaged._bind.built_for == nsa_build.bind_target()


def test_the_package_imports_where_torch_has_no_cuda():
    # as a torch that was built without CUDA: importing needs no device and no CUDA binding, and
    # the calls refuse host tensors by name
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import block_sparse_attention_selected_b200 as nsa
i = torch.zeros(1, dtype=torch.int32)
try:
    nsa.nsa_sel_paged_plan(i, i, i, i.view(1, 1), 16, 1)
except ValueError as e:
    assert "CUDA tensor" in str(e)
else:
    raise SystemExit("not refused")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(nsa.__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)
