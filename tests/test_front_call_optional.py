"""The operators in front of the projections without their native call path, and with a module that has only the gated
feed-forward operators' (CPU only)."""

import os
import subprocess
import sys

import pytest

from tests.test_native_call_optional import _package

USE = """
import sys, types
import torch
if {old}:
    old = types.ModuleType("precision_fp8_quant_amd._ffn_call")
    old.torch_version = torch.__version__.split("+")[0]
    sys.modules["precision_fp8_quant_amd._ffn_call"] = old
import precision_fp8_quant_amd as fp8q
from precision_fp8_quant_amd import ffn, front
assert fp8q.__file__.startswith({root!r}), fp8q.__file__
assert (ffn._native is not None) == {old} and front._native is None
f, i, u = torch.ones((4, 128)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 128), dtype=torch.uint8)
for call in (lambda: fp8q.fp8_rmsnorm(f, f[0]), lambda: fp8q.int8_rmsnorm(f, f[0]), lambda: fp8q.moe_route(f, 2),
             lambda: fp8q.rmsnorm_backward(f, f, f[0], f[:, 0]), lambda: fp8q.moe_route_backward(f, i),
             lambda: fp8q.fp8_moe_dispatch(i, u, f[:1, :4], 8)):
    try:
        call()
    except ValueError as e:
        assert "must be a device tensor" in str(e), e
    else:
        raise AssertionError("a host tensor was taken")
print("fine")
"""


@pytest.mark.parametrize("old", [False, True])
def test_calls_without_native_functions(tmp_path, old):
    dst = _package(tmp_path)
    if old:
        (dst / "_ffn_call.so").write_bytes(b"")
    res = subprocess.run([sys.executable, "-c", USE.format(root=str(tmp_path), old=old)], capture_output=True, text=True,
                         env=dict(os.environ, PYTHONPATH=str(tmp_path)), cwd=tmp_path, timeout=300)
    assert res.returncode == 0 and "fine" in res.stdout, res.stderr
