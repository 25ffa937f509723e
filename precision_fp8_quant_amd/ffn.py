"""Binding of the gated feed-forward operators (include/fp8q_ffn.h).

    fp8_gemm_gated(a, sa, b, sb, act)        -> h, or (h, gu) with save_gate_up=True
    fp8_gated_backward(dh, gu, act, mode)    -> (q, scales, q_t, scales_t)
    int8_quant_rows(x)                       -> (q, scales)
    int8_gemm(a, sa, b, sb, bias)            -> c
    int8_gemm_gated(a, sa, b, sb, act)       -> h
Argument marshalling only, like the package's other entry points.  Weights of
a gated projection are stacked: gate rows, then up rows.  8-bit integer
tensors are torch.int8 with rows a multiple of 16 bytes apart; outputs that
the binding allocates have such rows too, so a tensor whose last dimension is
no multiple of 16 bytes comes back as a view of wider rows.
"""

import ctypes
import os
import warnings

import torch

from . import BF16, F32, MAXABS, OK, _cdiv, _check, _codes, _expect, _i64, _int, _outputs_on, _ptr, _rowmajor, _run, lib

_NATIVE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_ffn_call.so")


def _load_native():
    """The native call path, or None where it was not built or was built for another torch: every call works without
    it, through ctypes and with more host time."""
    if not os.path.exists(_NATIVE_PATH):
        return None
    try:
        from . import _ffn_call
    except ImportError as e:
        why = str(e)
    else:
        if _ffn_call.torch_version == torch.__version__.split("+")[0]:
            return _ffn_call
        why = f"built for torch {_ffn_call.torch_version}, this is {torch.__version__}"
    warnings.warn(f"{_NATIVE_PATH} is not used: {why}. Rebuild it with __graft_entry__.build(); until then calls of the "
                  "gated feed-forward operators take more host time", RuntimeWarning, stacklevel=3)
    return None


_native = _load_native()

# enum of include/fp8q_ffn.h
ACT_SILU, ACT_GELU_TANH = 0, 1

# (name, argtypes) for every entry point of include/fp8q_ffn.h
SIGNATURES = {
    "fp8_gemm_gated": [_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _ptr, _i64, _ptr, _ptr, _int, _i64, _ptr, _i64,
                       _ptr],
    "fp8_gated_backward": [_int, _i64, _i64, _ptr, _i64, _ptr, _i64, _int, _int, _ptr, _i64, _ptr, _ptr, _i64, _ptr,
                           _ptr, _i64, _ptr],
    "int8_quant_rows": [_ptr, _int, _i64, _i64, _i64, _ptr, _i64, _ptr, _ptr],
    "int8_gemm": [_i64, _i64, _i64, _ptr, _i64, _ptr, _ptr, _i64, _ptr, _ptr, _ptr, _int, _i64, _ptr],
    "int8_gemm_gated": [_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _ptr, _i64, _ptr, _ptr, _int, _i64, _ptr],
}

for _name, _argtypes in SIGNATURES.items():
    getattr(lib, _name).argtypes = _argtypes
    getattr(lib, _name).restype = ctypes.c_int


# A caller with few tokens waits for the host rather than for the kernel.  The usual call (new outputs, current device
# and stream) is made by csrc/ffn/binding.cpp in one step; it answers None for anything else, and an int where the C ABI
# refuses.  What follows it here takes every call, and says what is wrong with one.
_bf16, _f32, _i8 = torch.bfloat16, torch.float32, torch.int8
_CODE = {_bf16: BF16, _f32: F32}


def _done(r):
    """The native call's answer: a result, or the C ABI's refusal as an error."""
    if r.__class__ is int:
        _check(r)
    return r


def _call(fn, dev, stream, *args):
    if stream is None and torch._C._cuda_getDevice() == dev.index:      # the current device's current stream
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
        if status != OK:
            _check(status)
    else:
        _run(fn, dev, stream, *args)


def _ld(t):
    """Leading dimension in elements; a single row's is its width in whole 16-byte chunks."""
    rows, cols = t.shape
    if rows > 1:
        return t.stride()[0]
    per = 16 // t.element_size()
    return max(cols + -cols % per, per)


def _dense(t, name, shape, device):
    """An FP32 array of scales or biases."""
    if not (t.dtype is _f32 and t.shape == shape and t.is_contiguous() and t.device == device and t.is_cuda):
        _expect(t, name, _f32, shape, device, dense=True)
    return t.data_ptr()


def _out(t, name, dtype, rows, cols, device):
    """The caller's output tensor, checked, or a new one; its dtype code and leading dimension."""
    if t is not None:
        dtype = t.dtype
    code = _CODE.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    if t is not None:
        _expect(t, name, dtype, (rows, cols), device)
        return t, code, _ld(t)
    pad = -cols % (8 if code == BF16 else 4)
    if pad:                                        # rows a multiple of 16 bytes apart
        return torch.empty_strided((rows, cols), (cols + pad, 1), dtype=dtype, device=device), code, cols + pad
    return torch.empty(rows, cols, dtype=dtype, device=device), code, cols or 1


def _ints(t, name):
    """Leading dimension of an 8-bit integer operand, whose rows the library reads in whole 16-byte chunks."""
    if not (t.dtype is _i8 and t.dim() == 2 and t.is_cuda):
        _rowmajor(t, name)
        raise TypeError(f"{name} must be torch.int8, got {t.dtype}")
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        _rowmajor(t, name)
    if rows <= 1:
        ld = max(cols + -cols % 16, 16)
    # any other leading dimension is the ABI's FP8Q_ERR_ALIGN
    if cols % 16 and rows and ld % 16 == 0:
        if t.storage_offset() + (rows - 1) * ld + cols + -cols % 16 > t.untyped_storage().nbytes():
            raise ValueError(f"{name}'s rows are read in whole 16-byte chunks: the storage must hold the last row up to "
                             "the next multiple of 16 bytes")
    return ld


def fp8_gemm_gated(a, a_scales, b, b_scales, act=ACT_SILU, out_dtype=torch.bfloat16, h=None, gu=None,
                   save_gate_up=False, stream=None):
    """h[M][F] = act(A Bg^T) * (A Bu^T) from block-scaled FP8 operands: a [M][K] in 1x128 tiles, b [2F][K] the stacked
    gate and up weights in 128x128 blocks.  With save_gate_up=True (or a gu tensor) also gu[M][2F], the
    pre-activations that fp8_gated_backward takes."""
    if _native and h is None and gu is None and stream is None:
        r = _native.fp8_gemm_gated(a, a_scales, b, b_scales, act, _CODE.get(out_dtype), save_gate_up)
        if r is not None:
            return _done(r)
    a, b = _codes(_rowmajor(a, "a")), _codes(_rowmajor(b, "b"))
    (m, k), (n2, kb), dev = a.shape, b.shape, a.device
    if kb != k:
        raise ValueError("a and b disagree on K")
    if n2 % 2:
        raise ValueError("b must hold as many gate rows as up rows")
    if b.device != dev:
        raise ValueError(f"b must be a tensor on {dev}")
    f, kg = n2 // 2, _cdiv(k, 128)
    sa = _dense(a_scales, "a_scales", (kg, m), dev)
    sb = _dense(b_scales, "b_scales", (_cdiv(n2, 128), kg), dev)
    gu_ptr, ldgu = None, 0
    with _outputs_on(stream, dev, h, gu if save_gate_up else h):
        h, code, ldh = _out(h, "h", out_dtype, m, f, dev)
        if gu is not None or save_gate_up:
            gu, gu_code, ldgu = _out(gu, "gu", h.dtype, m, n2, dev)
            if gu_code != code:
                raise TypeError(f"gu must be {h.dtype} like h, got {gu.dtype}")
            gu_ptr = gu.data_ptr()
    _call(lib.fp8_gemm_gated, dev, stream, act, m, f, k, a.data_ptr(), _ld(a), sa, b.data_ptr(), _ld(b), sb,
          h.data_ptr(), code, ldh, gu_ptr, ldgu)
    return h if gu is None else (h, gu)


def fp8_gated_backward(dh, gu, act=ACT_SILU, mode=MAXABS, q=None, scales=None, q_t=None, scales_t=None, dgu=None,
                       stream=None):
    """Gradient D = [dg | du] of h = act(g) * u from dh [M][F] and gu [M][2F] (both bf16 or both fp32), quantized in
    1x128 tiles (q [Mp][2F], scales [2F/128][Mp]: Dgrad's operand) and transposed 128x1 tiles (q_t [2F][Mp],
    scales_t [Mp/128][2F]: Wgrad's), Mp being M rounded up to whole 128-row tiles and the rows past M zero.  A dgu
    tensor [M][2F] also receives D itself."""
    if _native and q is None and scales is None and q_t is None and scales_t is None and dgu is None and stream is None:
        r = _native.fp8_gated_backward(dh, gu, act, mode)
        if r is not None:
            return _done(r)
    _rowmajor(dh, "dh")
    (m, f), dev, dtype = dh.shape, dh.device, dh.dtype
    code = _CODE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (bfloat16 or float32)")
    mp, f2 = m + -m % 128, 2 * f
    _expect(gu, "gu", dtype, (m, f2), dev)
    ds, ts = (f2 // 128, mp), (mp // 128, f2)      # F is a multiple of 128 or the ABI's FP8Q_ERR_UNSUPPORTED
    with _outputs_on(stream, dev, q, scales, q_t, scales_t):
        if q is None:
            q = torch.empty(mp, f2, dtype=torch.uint8, device=dev)
        if scales is None:
            scales = torch.empty(*ds, dtype=_f32, device=dev)
        if q_t is None:
            q_t = torch.empty(f2, mp, dtype=torch.uint8, device=dev)
        if scales_t is None:
            scales_t = torch.empty(*ts, dtype=_f32, device=dev)
    q, q_t = _expect(_codes(q), "q", torch.uint8, (mp, f2), dev), _expect(_codes(q_t), "q_t", torch.uint8, (f2, mp), dev)
    s, st = _dense(scales, "scales", ds, dev), _dense(scales_t, "scales_t", ts, dev)
    dgu_ptr, ld_dgu = None, 0
    if dgu is not None:
        _expect(dgu, "dgu", dtype, (m, f2), dev)
        dgu_ptr, ld_dgu = dgu.data_ptr(), _ld(dgu)
    _call(lib.fp8_gated_backward, dev, stream, act, m, f, dh.data_ptr(), _ld(dh), gu.data_ptr(), _ld(gu), code, mode,
          q.data_ptr(), _ld(q), s, q_t.data_ptr(), _ld(q_t), st, dgu_ptr, ld_dgu)
    return q, scales, q_t, scales_t


def int8_quant_rows(x, q=None, scales=None, stream=None):
    """Symmetric 8-bit codes of a 2-D bf16/fp32 tensor with one scale for each row (token or output channel):
    q int8 [rows][cols], scales [rows], x ~= q * scales[:, None]."""
    if _native and q is None and scales is None and stream is None:
        r = _native.int8_quant_rows(x)
        if r is not None:
            return _done(r)
    _rowmajor(x, "x")
    (rows, cols), dev = x.shape, x.device
    code = _CODE.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype} (bfloat16 or float32)")
    with _outputs_on(stream, dev, q, scales):
        if q is None:
            ld = max(cols + -cols % 16, 16)        # the last row's bytes up to 16 exist too, as int8_gemm reads them
            q = torch.empty(rows, ld, dtype=_i8, device=dev)
            if ld != cols:
                q = q.as_strided((rows, cols), (ld, 1))
        else:
            _expect(q, "q", _i8, (rows, cols), dev)
            ld = _ld(q)
        if scales is None:
            scales = torch.empty(rows, dtype=_f32, device=dev)
    _call(lib.int8_quant_rows, dev, stream, x.data_ptr(), code, rows, cols, _ld(x), q.data_ptr(), ld,
          _dense(scales, "scales", (rows,), dev))
    return q, scales


def int8_gemm(a, a_scales, b, b_scales, bias=None, out_dtype=torch.bfloat16, c=None, stream=None):
    """C[M][N] = a_scales[m] * b_scales[n] * (A . B^T) (+ bias[n]) from 8-bit integers a [M][K] and b [N][K]."""
    if _native and c is None and stream is None:
        r = _native.int8_gemm(a, a_scales, b, b_scales, bias, _CODE.get(out_dtype))
        if r is not None:
            return _done(r)
    lda, ldb = _ints(a, "a"), _ints(b, "b")
    (m, k), (n, kb), dev = a.shape, b.shape, a.device
    if kb != k:
        raise ValueError("a and b disagree on K")
    if b.device != dev:
        raise ValueError(f"b must be a tensor on {dev}")
    sa, sb = _dense(a_scales, "a_scales", (m,), dev), _dense(b_scales, "b_scales", (n,), dev)
    bias_ptr = None if bias is None else _dense(bias, "bias", (n,), dev)
    with _outputs_on(stream, dev, c):
        c, code, ldc = _out(c, "c", out_dtype, m, n, dev)
    _call(lib.int8_gemm, dev, stream, m, n, k, a.data_ptr(), lda, sa, b.data_ptr(), ldb, sb, bias_ptr, c.data_ptr(),
          code, ldc)
    return c


def int8_gemm_gated(a, a_scales, b, b_scales, act=ACT_SILU, out_dtype=torch.bfloat16, h=None, stream=None):
    """h[M][F] = act(g) * u with g and u the int8_gemm products of a [M][K] and the stacked gate and up weights
    b [2F][K]."""
    if _native and h is None and stream is None:
        r = _native.int8_gemm_gated(a, a_scales, b, b_scales, act, _CODE.get(out_dtype))
        if r is not None:
            return _done(r)
    lda, ldb = _ints(a, "a"), _ints(b, "b")
    (m, k), (n2, kb), dev = a.shape, b.shape, a.device
    if kb != k:
        raise ValueError("a and b disagree on K")
    if n2 % 2:
        raise ValueError("b must hold as many gate rows as up rows")
    if b.device != dev:
        raise ValueError(f"b must be a tensor on {dev}")
    sa, sb = _dense(a_scales, "a_scales", (m,), dev), _dense(b_scales, "b_scales", (n2,), dev)
    with _outputs_on(stream, dev, h):
        h, code, ldh = _out(h, "h", out_dtype, m, n2 // 2, dev)
    _call(lib.int8_gemm_gated, dev, stream, act, m, n2 // 2, k, a.data_ptr(), lda, sa, b.data_ptr(), ldb, sb,
          h.data_ptr(), code, ldh)
    return h
