"""build() in a process that has the package imported already: what it imports afterwards is the new library, in every
module (CPU only; the compilers are stand-ins that copy what was built before)."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "precision_fp8_quant_amd")

SCRIPT = """
import sys
import precision_fp8_quant_amd as old
import __graft_entry__ as g
g.build()
import precision_fp8_quant_amd as new
assert new is not old and new.lib is not old.lib
assert new.ffn.lib is new.lib, "the gated operators still call the library that was loaded before"
assert new.ffn._check is new._check and new.int8_gemm is new.ffn.int8_gemm
print("ok", new.__file__)
"""


def _stub(path, source):
    path.write_text(f'#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\ncp "{source}" "$2"\n')
    path.chmod(0o755)
    return str(path)


def test_build_replaces_every_module(tmp_path):
    libs = {n: os.path.join(PKG, n) for n in ("libfp8q.so", "_ffn_call.so")}
    if not all(map(os.path.exists, libs.values())):
        pytest.skip("not built")
    dst = tmp_path / "precision_fp8_quant_amd"
    dst.mkdir()
    (tmp_path / "tests" / "hip").mkdir(parents=True)
    shutil.copy(os.path.join(ROOT, "__graft_entry__.py"), tmp_path)
    for f in os.listdir(PKG):
        if f.endswith(".py") or f in libs:
            shutil.copy(os.path.join(PKG, f), dst / f)
    env = dict(os.environ, PYTHONPATH=str(tmp_path), HIPCC=_stub(tmp_path / "hipcc", libs["libfp8q.so"]),
               CXX=_stub(tmp_path / "c++", libs["_ffn_call.so"]))
    res = subprocess.run([sys.executable, "-c", SCRIPT], capture_output=True, text=True, env=env, cwd=tmp_path, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert f"ok {dst}" in res.stdout
