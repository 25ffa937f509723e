"""Argument validation of include/fp8q_ffn.h under the host sanitizers: abi_ffn.cpp is built with AddressSanitizer and
UndefinedBehaviorSanitizer by the host compiler, linked with stand-ins for the launchers, and driven from plain C with
adversarial sizes, leading dimensions and addresses."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "precision_fp8_quant_amd", "csrc")
CLIENT = os.path.join(ROOT, "tests", "c_client")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]


def test_ffn_validation_under_sanitizers(tmp_path):
    gxx, gcc = shutil.which("g++"), shutil.which("gcc")
    if gxx is None or gcc is None:
        pytest.skip("no host compiler")
    inc = [f"-I{ROOT}/include", f"-I{CSRC}", f"-I{ROCM}/include", "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for src, cc, std in ((os.path.join(CSRC, "ffn", "abi_ffn.cpp"), gxx, "-std=c++17"),
                         (os.path.join(CLIENT, "ffn_stub_launch.cpp"), gxx, "-std=c++17"),
                         (os.path.join(CLIENT, "ffn_abi_adversarial.c"), gcc, "-std=c11")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run([cc, std, "-Wall", "-Werror", *SAN, *inc, "-c", src, "-o", obj], check=True, capture_output=True,
                       text=True)
        objs.append(obj)
    exe = str(tmp_path / "ffn_abi_adversarial")
    subprocess.run([gxx, *SAN, *objs, "-o", exe], check=True, capture_output=True, text=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=env)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "adversarial validation ok (8 launches reached)" in res.stdout
    assert "runtime error" not in res.stderr and "ERROR: AddressSanitizer" not in res.stderr
