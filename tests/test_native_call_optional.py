"""The native call path of the gated feed-forward operators (_ffn_call.so) is an extra: without it, or with one that
was built for another torch, the package imports and every call goes through ctypes; and libfp8q.so builds with hipcc
alone, where there is no torch and no host compiler (CPU only)."""

import os
import shutil
import stat
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "precision_fp8_quant_amd")
BUILD = os.path.join(PKG, "_build.py")
LIB = os.path.join(PKG, "libfp8q.so")

USE = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import precision_fp8_quant_amd as fp8q
import torch
from precision_fp8_quant_amd import ffn
assert fp8q.__file__.startswith({root!r}), fp8q.__file__
assert ffn._native is None
assert fp8q.lib.fp8q_abi_version() > 0
assert fp8q.lib.int8_gemm(0, 1, 1, None, 0, None, None, 0, None, None, None, fp8q.BF16, 0, None) == fp8q.OK
i8, s = torch.zeros((4, 32), dtype=torch.int8), torch.ones(4)
bf = torch.zeros((4, 128), dtype=torch.bfloat16)
for call in (lambda: fp8q.int8_gemm(i8, s, i8, s), lambda: fp8q.int8_gemm_gated(i8, s, i8, s),
             lambda: fp8q.int8_quant_rows(s.view(2, 2)), lambda: fp8q.fp8_gated_backward(bf, bf),
             lambda: fp8q.fp8_gemm_gated(i8.view(torch.uint8), s, i8.view(torch.uint8), s)):
    try:
        call()
    except ValueError as e:
        assert "must be a device tensor" in str(e), e
    else:
        raise AssertionError("a host tensor was taken")
print("warned:", *[str(w.message) for w in seen if issubclass(w.category, RuntimeWarning)])
"""


def _package(tmp_path):
    """A copy of the package's Python files beside its C library, without the native call path."""
    if not os.path.exists(LIB):
        pytest.skip("libfp8q.so not built")
    dst = tmp_path / "precision_fp8_quant_amd"
    dst.mkdir()
    for f in os.listdir(PKG):
        if f.endswith(".py"):
            shutil.copy(os.path.join(PKG, f), dst / f)
    os.symlink(LIB, dst / "libfp8q.so")
    return dst


def _use(tmp_path, before=""):
    env = dict(os.environ, PYTHONPATH=str(tmp_path))
    res = subprocess.run([sys.executable, "-c", before + USE.format(root=str(tmp_path))], capture_output=True, text=True, env=env,
                         cwd=tmp_path, timeout=300)
    assert res.returncode == 0, res.stderr
    return res.stdout


def test_package_without_the_native_call_path(tmp_path):
    _package(tmp_path)
    assert _use(tmp_path).strip() == "warned:"


def test_package_with_an_unloadable_native_call_path(tmp_path):
    (_package(tmp_path) / "_ffn_call.so").write_text("no shared object")
    assert "_ffn_call.so is not used" in _use(tmp_path)


def test_package_with_a_native_call_path_for_another_torch(tmp_path):
    (_package(tmp_path) / "_ffn_call.so").write_text("")      # its stand-in is loaded already
    loaded = ("import sys, types; m = types.ModuleType('precision_fp8_quant_amd._ffn_call'); m.torch_version = '1.0.0'\n"
              "sys.modules[m.__name__] = m\n")
    assert "built for torch 1.0.0" in _use(tmp_path, loaded)


BUILD_ALONE = """
import importlib.util, os, sys
{before}
spec = importlib.util.spec_from_file_location("_b", {build!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.BUILD_DIR, b.LIB_PATH, b.BINDING_PATH = {tmp!r} + "/o", {tmp!r} + "/libfp8q.so", {tmp!r} + "/_ffn_call.so"
try:
    b.build()
except RuntimeError as e:
    print("build failed:", str(e).splitlines()[0])
print("library", os.path.exists(b.LIB_PATH), "native", os.path.exists(b.BINDING_PATH))
"""


def _stub(path, body):
    path.write_text("#!/bin/sh\n" + body)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


def _build_alone(tmp_path, before, cxx):
    hipcc = _stub(tmp_path / "hipcc", 'while [ "$1" != -o ]; do shift; done\n: > "$2"\n')      # only writes its output
    res = subprocess.run([sys.executable, "-c", BUILD_ALONE.format(before=before, build=BUILD, tmp=str(tmp_path))],
                         capture_output=True, text=True, timeout=300, cwd=tmp_path,
                         env=dict(os.environ, HIPCC=hipcc, CXX=cxx))
    assert res.returncode == 0, res.stderr
    return res.stdout


def test_library_builds_without_torch(tmp_path):
    out = _build_alone(tmp_path, "sys.modules['torch'] = None", "/nonexistent/c++")
    assert "library True native False" in out and "build failed" not in out


def test_library_is_complete_when_the_native_call_path_fails_to_build(tmp_path):
    out = _build_alone(tmp_path, "", _stub(tmp_path / "c++", "exit 1\n"))
    assert "build failed: command failed (1)" in out and "library True native False" in out
