"""The marshalling module is a help for short calls, not a condition: the library is built and loaded
without it, and a module that does not fit the running torch or Python is made again."""
import os
import subprocess
import sys
import types

import pytest
import torch

import speculative_decoding_verification_token_gb300 as sv
from speculative_decoding_verification_token_gb300 import build as b


@pytest.fixture
def compiler(monkeypatch, tmp_path):
    """The host compiler replaced: `compiler.answer(cmd)` runs in its place; `compiler.runs` counts."""
    c = types.SimpleNamespace(runs=0, answer=None)

    def ok(cmd):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def run(cmd, **kw):
        c.runs += 1
        return c.answer(cmd)

    c.answer = c.ok = ok
    monkeypatch.setattr(b, "FASTCALL", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(b.subprocess, "run", run)
    return c


def _no_headers(cmd):
    return subprocess.CompletedProcess(cmd, 1, "", "fatal error: Python.h: No such file or directory")


def _no_compiler(cmd):
    raise FileNotFoundError(cmd[0])


@pytest.mark.parametrize("failure", [_no_headers, _no_compiler])
def test_library_is_built_without_the_module(compiler, failure, monkeypatch):
    monkeypatch.setattr(b, "build_library", lambda force, verbose: "library")
    assert b.build() == "library" and os.path.exists(b.FASTCALL)
    compiler.answer = failure
    with pytest.warns(RuntimeWarning, match="Python.h|c\\+\\+|g\\+\\+"):
        assert b.build(force=True) == "library"
    assert not os.path.exists(b.FASTCALL)  # the one before does not stay in its place
    compiler.answer = compiler.ok
    assert b.build() == "library" and os.path.exists(b.FASTCALL)


def test_made_again_for_another_torch_or_other_flags(compiler, monkeypatch):
    b.build_fastcall()
    b.build_fastcall()
    assert compiler.runs == 1
    monkeypatch.setattr(torch, "__version__", "0.0")
    b.build_fastcall()
    b.build_fastcall()
    assert compiler.runs == 2
    monkeypatch.setattr(b, "INCLUDE", b.INCLUDE + os.sep)
    b.build_fastcall()
    assert compiler.runs == 3


def test_what_is_built_needs_no_toolkit(monkeypatch):
    b.build()
    made = os.path.getmtime(b.FASTCALL)
    if os.path.exists("/usr/local/cuda/bin/nvcc"):  # the path the module was made with
        def none():
            raise RuntimeError("nvcc not found")
        monkeypatch.setattr(b, "_nvcc", none)
        assert b.build() == b.LIB and os.path.getmtime(b.FASTCALL) == made


def test_named_for_the_python_it_is_built_for():
    import sysconfig
    assert b.FASTCALL.endswith("_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))


def test_library_is_loaded_without_the_module(monkeypatch):
    b.build()
    sv.lib()
    monkeypatch.setattr(sv, "_lib", None)
    monkeypatch.setattr(sv, "_fast", None)
    monkeypatch.delattr(sv, "_fastcall", raising=False)
    monkeypatch.setitem(sys.modules, sv.__name__ + "._fastcall", None)  # importing it fails
    with pytest.warns(RuntimeWarning, match="_fastcall"):
        assert "sm_103a" in sv.version()
    assert sv._fast is None
    with pytest.raises(ValueError):  # the Python checks answer
        sv.spec_quantize_fp4(torch.zeros((2, 64)), sv.SV_FP4_E8M0_32)
