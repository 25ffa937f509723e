"""Compile the fp8q HIP library (libfp8q.so) and its native call path (_ffn_call.so) in-tree for gfx950.

Every kernel is hand-written HIP for CDNA4; this only drives hipcc.  The
library is linked into ``precision_fp8_quant_amd/libfp8q.so`` next to the
binding, so it travels with the source tree.
"""

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG_DIR), "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libfp8q.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

DEVICE_SOURCES = ["quant.hip", "gemm.hip", "gemm_pow2.hip", "ffn/fp8_gated.hip", "ffn/int8_gemm.hip",
                  "ffn/int8_quant.hip", "ffn/gated_backward.hip"]
HOST_SOURCES = ["abi.cpp", "ffn/abi_ffn.cpp"]

# -ffp-contract=off: the quantizer's scale-multiply-then-round sequence must be
# exactly the stated FP32 operations (no fused multiply-add formed behind our
# back); the GEMM asks for its FMAs explicitly.
# -packed-fp32-ops off: keep the compiler from forming packed FP32 VALU ops.
COMMON_FLAGS = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-I", INCLUDE, "-I", CSRC]
DEVICE_FLAGS = ["--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                "-Wno-unused-command-line-argument"]
# -amdgpu-mfma-vgpr-form: MFMA results go straight to VGPRs, where the FP32
# promotion FMAs read them (no v_accvgpr_read copies).  Not for the
# hardware-scaled GEMM, whose accumulators stay in AGPRs inside the MFMA chain.
PER_SOURCE_FLAGS = {"gemm.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
                    "ffn/fp8_gated.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


# The native call path of ffn.py: a CPython extension against torch's headers,
# linked to libfp8q.so beside it.  The package works without it.
BINDING_SRC = os.path.join(CSRC, "ffn", "binding.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_ffn_call.so")


def _binding_command(out):
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
            "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(rocm, "include"), BINDING_SRC, "-o", out]


def _link_binding(obj, verbose):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, "-L", libs, "-ltorch", "-ltorch_cpu", "-ltorch_python",
          "-lc10", "-lc10_hip", "-L", PKG_DIR, "-lfp8q", "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(tmp, BINDING_PATH)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"command failed ({res.returncode}): {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return res


def build_library(verbose=False, extra_flags=()):
    """Compile every source and link libfp8q.so, which needs nothing but hipcc."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = []
    for src in DEVICE_SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace("/", "_") + ".o")
        jobs.append([HIPCC, *COMMON_FLAGS, *DEVICE_FLAGS, *PER_SOURCE_FLAGS.get(src, []), *extra_flags,
                     "-c", os.path.join(CSRC, src), "-o", obj])
    for src in HOST_SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace("/", "_") + ".o")
        jobs.append([HIPCC, *COMMON_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj])
    objs = [j[-1] for j in jobs]
    with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
        list(ex.map(lambda c: _run(c, verbose), jobs))
    tmp = LIB_PATH + ".tmp"
    _run([HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *objs, "-o", tmp], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build(verbose=False, extra_flags=()):
    """libfp8q.so and, where torch is installed, the native call path (always recompiles).  The library is complete
    when the call path fails to build, which is still an error."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    binding = os.path.join(BUILD_DIR, "ffn_binding.cpp.o")
    with ThreadPoolExecutor(max_workers=1) as ex:  # beside the library's sources
        try:
            compiled = ex.submit(_run, _binding_command(binding), verbose)
        except ImportError as e:
            compiled = None
            print(f"{os.path.basename(BINDING_PATH)} is not built: {e}", flush=True)
        build_library(verbose, extra_flags)
    if compiled:
        compiled.result()
        _link_binding(binding, verbose)
    return LIB_PATH


TEST_PROBE_SRC = os.path.join(os.path.dirname(PKG_DIR), "tests", "hip", "scale_div_probe.hip")
TEST_PROBE_LIB = os.path.join(os.path.dirname(PKG_DIR), "tests", "hip", "libfp8q_divprobe.so")


def build_test_probe(verbose=False):
    """Compile the GPU test helper tests/hip/scale_div_probe.hip (not part of libfp8q.so) with the library's
    device flags, so that it exercises the same code as the quantizers."""
    tmp = TEST_PROBE_LIB + ".tmp"
    _run([HIPCC, *COMMON_FLAGS, *DEVICE_FLAGS, "-shared", TEST_PROBE_SRC, "-o", tmp], verbose)
    os.replace(tmp, TEST_PROBE_LIB)
    return TEST_PROBE_LIB


if __name__ == "__main__":
    print(build(verbose=True))
