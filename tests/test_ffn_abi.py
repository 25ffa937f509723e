"""include/fp8q_ffn.h: every entry point is exported and bound, arguments are rejected before anything is launched, and
the 64-bit definitions of oracle/ffn.py hold against differences (CPU only: no call here reaches a kernel launch)."""

import ctypes
import os
import re

import numpy as np
import pytest

from oracle import ffn as of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8q_ffn.h")

fp8q = pytest.importorskip("precision_fp8_quant_amd", reason="libfp8q.so not built")
from precision_fp8_quant_amd import ffn  # noqa: E402

A, B, C, D = 0x10000000, 0x20000000, 0x40000000, 0x60000000    # fake 16-byte aligned device addresses
E, G = 0x70000000, 0x78000000
HUGE = 1 << 62


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(ffn.SIGNATURES) == {"fp8_gemm_gated", "fp8_gated_backward", "int8_quant_rows", "int8_gemm",
                                            "int8_gemm_gated"}
    raw = ctypes.CDLL(fp8q.LIB_PATH)
    for n in names:
        assert hasattr(raw, n) and callable(getattr(fp8q, n)), n


def _gated(**kw):
    v = dict(act=0, m=100, f=256, k=384, a=A, lda=384, sa=B, b=C, ldb=384, sb=D, h=E, dt=fp8q.BF16, ldh=256, gu=None,
             ldgu=0)
    v.update(kw)
    return fp8q.lib.fp8_gemm_gated(v["act"], v["m"], v["f"], v["k"], v["a"], v["lda"], v["sa"], v["b"], v["ldb"],
                                   v["sb"], v["h"], v["dt"], v["ldh"], v["gu"], v["ldgu"], None)


@pytest.mark.parametrize("want, kw", [
    ("OK", dict(m=0, a=None)), ("OK", dict(f=0, h=None)),
    ("ERR_ARG", dict(act=2)), ("ERR_ARG", dict(act=-1)), ("ERR_ARG", dict(dt=2)),
    ("ERR_SHAPE", dict(m=-1)), ("ERR_SHAPE", dict(k=-128)), ("ERR_SHAPE", dict(f=HUGE + 128, ldh=HUGE + 128)),
    ("ERR_NULL", dict(h=None)), ("ERR_NULL", dict(a=None)), ("ERR_NULL", dict(sb=None)),
    ("ERR_SHAPE", dict(lda=368)), ("ERR_SHAPE", dict(ldb=0)), ("ERR_SHAPE", dict(ldh=248)),
    ("ERR_SHAPE", dict(gu=G, ldgu=504)),
    ("ERR_ALIGN", dict(a=A + 8)), ("ERR_ALIGN", dict(ldb=392)), ("ERR_ALIGN", dict(ldh=260)),
    ("ERR_ALIGN", dict(gu=G + 2, ldgu=512)), ("ERR_ALIGN", dict(sa=B + 4)),
    ("ERR_UNSUPPORTED", dict(f=192)), ("ERR_UNSUPPORTED", dict(k=320)),
    ("ERR_UNSUPPORTED", dict(lda=1 << 22)), ("ERR_UNSUPPORTED", dict(m=1 << 40)),
    ("ERR_ALIAS", dict(h=A + 384)), ("ERR_ALIAS", dict(gu=E + 256, ldgu=512)), ("ERR_ALIAS", dict(gu=D, ldgu=512)),
])
def test_gemm_gated_validation(want, kw):
    assert _gated(**kw) == getattr(fp8q, want), kw


def _bwd(**kw):
    v = dict(act=1, m=200, f=256, dh=A, lddh=256, gu=B, ldgu=512, dt=fp8q.BF16, mode=0, q=C, ldq=512, s=D, qt=E,
             ldqt=256, st=G, dgu=None, lddgu=0)
    v.update(kw)
    return fp8q.lib.fp8_gated_backward(v["act"], v["m"], v["f"], v["dh"], v["lddh"], v["gu"], v["ldgu"], v["dt"],
                                       v["mode"], v["q"], v["ldq"], v["s"], v["qt"], v["ldqt"], v["st"], v["dgu"],
                                       v["lddgu"], None)


@pytest.mark.parametrize("want, kw", [
    ("OK", dict(m=0, dh=None)), ("OK", dict(f=0, q=None)),
    ("ERR_ARG", dict(act=7)), ("ERR_ARG", dict(dt=-1)), ("ERR_ARG", dict(mode=2)),
    ("ERR_SHAPE", dict(m=-5)), ("ERR_SHAPE", dict(f=HUGE)), ("ERR_SHAPE", dict(m=(1 << 63) - 1)),
    *[("ERR_NULL", {n: None}) for n in ("dh", "gu", "q", "s", "qt", "st")],
    ("ERR_SHAPE", dict(lddh=128)), ("ERR_SHAPE", dict(ldgu=256)), ("ERR_SHAPE", dict(ldq=256)),
    ("ERR_SHAPE", dict(ldqt=208)),                     # q_t holds whole 128-row tiles: 256 columns for 200 rows
    ("ERR_SHAPE", dict(dgu=0x7C000000, lddgu=256)),
    ("ERR_ALIGN", dict(dh=A + 2)), ("ERR_ALIGN", dict(ldqt=264)), ("ERR_ALIGN", dict(st=G + 4)),
    ("ERR_ALIGN", dict(dgu=0x7C000000, lddgu=516)),
    ("ERR_UNSUPPORTED", dict(f=160)),
    ("ERR_ALIAS", dict(q=A + 256)), ("ERR_ALIAS", dict(q=B + 200 * 512)), ("ERR_ALIAS", dict(st=D + 16)),
    ("ERR_ALIAS", dict(q=A - 255 * 512)),              # the padded rows of q reach into dh
    ("ERR_ALIAS", dict(dgu=B, lddgu=512)),
])
def test_gated_backward_validation(want, kw):
    assert _bwd(**kw) == getattr(fp8q, want), kw


def _quant(**kw):
    v = dict(x=A, dt=fp8q.BF16, rows=7, cols=1001, ldx=1008, q=B, ldq=1008, s=C)
    v.update(kw)
    return fp8q.lib.int8_quant_rows(v["x"], v["dt"], v["rows"], v["cols"], v["ldx"], v["q"], v["ldq"], v["s"], None)


@pytest.mark.parametrize("want, kw", [
    ("OK", dict(rows=0, x=None)),
    ("ERR_ARG", dict(dt=2)), ("ERR_SHAPE", dict(cols=-1)), ("ERR_SHAPE", dict(rows=-1)),
    ("ERR_NULL", dict(x=None)), ("ERR_NULL", dict(q=None)), ("ERR_NULL", dict(s=None)), ("ERR_NULL", dict(cols=0, s=None)),
    ("ERR_SHAPE", dict(ldx=1000)), ("ERR_SHAPE", dict(ldq=992)),
    ("ERR_ALIGN", dict(ldx=1001)), ("ERR_ALIGN", dict(ldq=1001)), ("ERR_ALIGN", dict(x=A + 4)),
    ("ERR_ALIAS", dict(q=A)), ("ERR_ALIAS", dict(s=B + 1008)),
    ("ERR_SHAPE", dict(rows=HUGE, ldx=HUGE)),
])
def test_int8_quant_validation(want, kw):
    assert _quant(**kw) == getattr(fp8q, want), kw


def _int8(gated, **kw):
    v = dict(act=0, m=5, n=37, k=1001, a=A, lda=1008, sa=B, b=C, ldb=1008, sb=D, bias=None, c=E, dt=fp8q.F32, ldc=40)
    v.update(kw)
    if gated:
        return fp8q.lib.int8_gemm_gated(v["act"], v["m"], v["n"], v["k"], v["a"], v["lda"], v["sa"], v["b"], v["ldb"],
                                        v["sb"], v["c"], v["dt"], v["ldc"], None)
    return fp8q.lib.int8_gemm(v["m"], v["n"], v["k"], v["a"], v["lda"], v["sa"], v["b"], v["ldb"], v["sb"], v["bias"],
                              v["c"], v["dt"], v["ldc"], None)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("want, kw", [
    ("OK", dict(m=0, a=None)), ("OK", dict(n=0, c=None)),
    ("ERR_ARG", dict(dt=5)),
    ("ERR_SHAPE", dict(n=-1)), ("ERR_SHAPE", dict(k=-1)),
    ("ERR_NULL", dict(c=None)), ("ERR_NULL", dict(b=None)), ("ERR_NULL", dict(sa=None)),
    ("ERR_SHAPE", dict(lda=992)), ("ERR_SHAPE", dict(ldc=36)),
    ("ERR_ALIGN", dict(lda=1001)), ("ERR_ALIGN", dict(ldc=38)), ("ERR_ALIGN", dict(b=C + 1)), ("ERR_ALIGN", dict(sb=D + 8)),
    ("ERR_UNSUPPORTED", dict(k=131057, lda=131072, ldb=131072)),     # the 32-bit sum could overflow
    ("ERR_UNSUPPORTED", dict(ldb=1 << 22)),
    ("ERR_UNSUPPORTED", dict(m=1 << 40, n=1 << 20, ldc=1 << 20)),
    ("ERR_ALIAS", dict(c=A)), ("ERR_ALIAS", dict(c=C + 36 * 1008 + 1000 - 1000 % 16 + 0)), ("ERR_ALIAS", dict(sa=E + 64)),
])
def test_int8_product_validation(want, kw, gated):
    assert _int8(gated, **kw) == getattr(fp8q, want), kw


def test_int8_bias_and_act_validation():
    assert _int8(False, bias=G + 4) == fp8q.ERR_ALIGN
    assert _int8(False, bias=E + 128) == fp8q.ERR_ALIAS
    assert _int8(True, act=2) == fp8q.ERR_ARG
    assert _int8(True, n=HUGE, ldc=HUGE) == fp8q.ERR_SHAPE           # 2F overflows


# --- the definitions themselves -------------------------------------------

@pytest.mark.parametrize("kind", [of.SILU, of.GELU_TANH])
def test_slope_against_differences(kind):
    """act'(g) against central differences: with step 1e-5 the truncation (third derivative under 2) is under 4e-11
    and the rounding of values up to 30 under 30 * 2^-52 / 1e-5 = 7e-10."""
    g = np.linspace(-30, 30, 6001)
    d = (of.act(g + 1e-5, kind) - of.act(g - 1e-5, kind)) / ((g + 1e-5) - (g - 1e-5))
    assert np.max(np.abs(d - of.act_slope(g, kind))) <= 1e-9


def test_activations_against_their_textbook_forms():
    """GELU's tanh form and SiLU's quotient, within the rounding of values up to 12."""
    g = np.linspace(-12, 12, 2001)
    z = np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    assert np.max(np.abs(of.act(g, of.GELU_TANH) - 0.5 * g * (1 + np.tanh(z)))) <= 1e-14
    assert np.max(np.abs(of.act(g, of.SILU) - g / (1 + np.exp(-g)))) <= 1e-14


def test_int8_codes_of_a_worked_row():
    """a = 254 gives s = 2 and inv = 0.5 exactly: halves round to even, the largest value to 127."""
    q, s = of.quant_int8_rows(np.array([[254, 1, 3, 5, -1, -3, -254, 0]], np.float32))
    assert s[0] == 2.0 and q.tolist() == [[127, 0, 2, 2, 0, -2, -127, 0]]
    q, s = of.quant_int8_rows(np.zeros((1, 3), np.float32))
    assert s[0] == np.float32(2.0 ** -126) and not q.any()


def test_native_call_leaves_unusual_calls_to_the_binding():
    """What the native call path does not expect it leaves alone (None): ffn.py then names what is wrong."""
    import torch
    from precision_fp8_quant_amd import _ffn_call as native
    i8, s = torch.zeros((4, 32), dtype=torch.int8), torch.ones(4)
    assert native.int8_gemm(i8, s, i8, s, None, fp8q.BF16) is None                 # host tensors
    assert native.int8_gemm(1, None, "a", s, 2.5, 1 << 80) is None
    assert native.int8_gemm() is None and native.fp8_gated_backward(i8) is None
    assert native.int8_gemm_gated(i8, s, i8, s, -1, fp8q.BF16) is None
    assert native.fp8_gemm_gated(i8, s, i8, s, 0, 0, 1) is None
    assert native.int8_quant_rows(s) is None
    with pytest.raises(ValueError, match="must be a device tensor"):
        fp8q.int8_gemm(i8, s, i8, s)
