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

import torch

from . import BF16, F32, MAXABS, _cdiv, _codes, _dtype_code, _expect, _i64, _int, _ptr, _rowmajor, _run, lib

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


def _ld(t):
    """Leading dimension in elements; a single row's is its width in whole 16-byte chunks."""
    rows, cols = t.shape
    if rows > 1:
        return t.stride(0)
    per = 16 // t.element_size()
    return max(cols + -cols % per, per)


_OUT_CODE = {torch.bfloat16: BF16, torch.float32: F32}


def _out(t, name, dtype, rows, cols, device):
    """The caller's output tensor, checked, or a new one; its dtype code and leading dimension."""
    if t is not None:
        dtype = t.dtype
    code = _OUT_CODE.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    if t is None:
        pad = -cols % (16 // dtype.itemsize)
        t = torch.empty((rows, cols + pad), dtype=dtype, device=device)
        return (t[:, :cols] if pad else t), code, max(cols + pad, 1)
    _expect(t, name, dtype, (rows, cols), device)
    return t, code, _ld(t)


def _ints(t, name):
    """Leading dimension of an 8-bit integer operand, whose rows the library reads in whole 16-byte chunks."""
    if t.dtype is torch.int8 and t.dim() == 2 and t.is_cuda:
        rows, cols = t.shape
        if cols % 16 == 0 and cols and t.stride(1) == 1:       # no chunk reaches beyond a row
            return t.stride(0) if rows > 1 else cols
    _rowmajor(t, name)
    if t.dtype != torch.int8:
        raise TypeError(f"{name} must be torch.int8, got {t.dtype}")
    rows, cols = t.shape
    ld = _ld(t)
    # any other leading dimension is the ABI's FP8Q_ERR_ALIGN
    if rows and cols and ld % 16 == 0:
        if t.storage_offset() + (rows - 1) * ld + cols + -cols % 16 > t.untyped_storage().nbytes():
            raise ValueError(f"{name}'s rows are read in whole 16-byte chunks: the storage must hold the last row up to "
                             "the next multiple of 16 bytes")
    return ld


def fp8_gemm_gated(a, a_scales, b, b_scales, act=ACT_SILU, out_dtype=torch.bfloat16, h=None, gu=None,
                   save_gate_up=False, stream=None):
    """h[M][F] = act(A Bg^T) * (A Bu^T) from block-scaled FP8 operands: a [M][K] in 1x128 tiles, b [2F][K] the stacked
    gate and up weights in 128x128 blocks.  With save_gate_up=True (or a gu tensor) also gu[M][2F], the
    pre-activations that fp8_gated_backward takes."""
    a, b = _codes(_rowmajor(a, "a")), _codes(_rowmajor(b, "b"))
    (m, k), (n2, dev) = a.shape, (b.shape[0], a.device)
    if b.shape[1] != k:
        raise ValueError("a and b disagree on K")
    if n2 % 2:
        raise ValueError("b must hold as many gate rows as up rows")
    f = n2 // 2
    _expect(b, "b", torch.uint8, (n2, k), dev)
    _expect(a_scales, "a_scales", torch.float32, (_cdiv(k, 128), m), dev, dense=True)
    _expect(b_scales, "b_scales", torch.float32, (_cdiv(n2, 128), _cdiv(k, 128)), dev, dense=True)
    h, code, ldh = _out(h, "h", out_dtype, m, f, dev)
    gu_ptr, ldgu = None, 0
    if gu is not None or save_gate_up:
        gu, gu_code, ldgu = _out(gu, "gu", h.dtype, m, n2, dev)
        if gu_code != code:
            raise TypeError(f"gu must be {h.dtype} like h, got {gu.dtype}")
        gu_ptr = gu.data_ptr()
    _run(lib.fp8_gemm_gated, dev, stream, act, m, f, k, a.data_ptr(), _ld(a), a_scales.data_ptr(), b.data_ptr(),
         _ld(b), b_scales.data_ptr(), h.data_ptr(), code, ldh, gu_ptr, ldgu)
    return h if gu is None else (h, gu)


def fp8_gated_backward(dh, gu, act=ACT_SILU, mode=MAXABS, q=None, scales=None, q_t=None, scales_t=None, dgu=None,
                       stream=None):
    """Gradient D = [dg | du] of h = act(g) * u from dh [M][F] and gu [M][2F] (both bf16 or both fp32), quantized in
    1x128 tiles (q [Mp][2F], scales [2F/128][Mp]: Dgrad's operand) and transposed 128x1 tiles (q_t [2F][Mp],
    scales_t [Mp/128][2F]: Wgrad's), Mp being M rounded up to whole 128-row tiles and the rows past M zero.  A dgu
    tensor [M][2F] also receives D itself."""
    _rowmajor(dh, "dh")
    m, f = dh.shape
    dev, mp, f2 = dh.device, _cdiv(dh.shape[0], 128) * 128, 2 * dh.shape[1]
    _expect(gu, "gu", dh.dtype, (m, f2), dev)
    ds, ts = (f2 // 128, mp), (mp // 128, f2)      # F is a multiple of 128 or the ABI's FP8Q_ERR_UNSUPPORTED
    if q is None:
        q = torch.empty((mp, f2), dtype=torch.uint8, device=dev)
    else:
        q = _expect(_codes(q), "q", torch.uint8, (mp, f2), dev)
    if scales is None:
        scales = torch.empty(ds, dtype=torch.float32, device=dev)
    else:
        _expect(scales, "scales", torch.float32, ds, dev, dense=True)
    if q_t is None:
        q_t = torch.empty((f2, mp), dtype=torch.uint8, device=dev)
    else:
        q_t = _expect(_codes(q_t), "q_t", torch.uint8, (f2, mp), dev)
    if scales_t is None:
        scales_t = torch.empty(ts, dtype=torch.float32, device=dev)
    else:
        _expect(scales_t, "scales_t", torch.float32, ts, dev, dense=True)
    if dgu is not None:
        _expect(dgu, "dgu", dh.dtype, (m, f2), dev)
    _run(lib.fp8_gated_backward, dev, stream, act, m, f, dh.data_ptr(), _ld(dh), gu.data_ptr(), _ld(gu),
         _dtype_code(dh), mode, q.data_ptr(), _ld(q), scales.data_ptr(), q_t.data_ptr(), _ld(q_t),
         scales_t.data_ptr(), None if dgu is None else dgu.data_ptr(), 0 if dgu is None else _ld(dgu))
    return q, scales, q_t, scales_t


def int8_quant_rows(x, q=None, scales=None, stream=None):
    """Symmetric 8-bit codes of a 2-D bf16/fp32 tensor with one scale for each row (token or output channel):
    q int8 [rows][cols], scales [rows], x ~= q * scales[:, None]."""
    _rowmajor(x, "x")
    rows, cols = x.shape
    dev = x.device
    if q is None:
        ld = max(cols + -cols % 16, 16)
        q = torch.empty((rows, ld), dtype=torch.int8, device=dev)
        if ld != cols:
            q = q[:, :cols]
    else:
        _expect(q, "q", torch.int8, (rows, cols), dev)
        ld = _ld(q)
    if scales is None:
        scales = torch.empty((rows,), dtype=torch.float32, device=dev)
    else:
        _expect(scales, "scales", torch.float32, (rows,), dev, dense=True)
    _run(lib.int8_quant_rows, dev, stream, x.data_ptr(), _dtype_code(x), rows, cols, _ld(x), q.data_ptr(), ld,
         scales.data_ptr())
    return q, scales


def int8_gemm(a, a_scales, b, b_scales, bias=None, out_dtype=torch.bfloat16, c=None, stream=None):
    """C[M][N] = a_scales[m] * b_scales[n] * (A . B^T) (+ bias[n]) from 8-bit integers a [M][K] and b [N][K]."""
    lda, ldb = _ints(a, "a"), _ints(b, "b")
    (m, k), n, dev = a.shape, b.shape[0], a.device
    if b.shape[1] != k:
        raise ValueError("a and b disagree on K")
    _expect(b, "b", torch.int8, (n, k), dev)
    _expect(a_scales, "a_scales", torch.float32, (m,), dev, dense=True)
    _expect(b_scales, "b_scales", torch.float32, (n,), dev, dense=True)
    if bias is not None:
        _expect(bias, "bias", torch.float32, (n,), dev, dense=True)
    c, code, ldc = _out(c, "c", out_dtype, m, n, dev)
    _run(lib.int8_gemm, dev, stream, m, n, k, a.data_ptr(), lda, a_scales.data_ptr(), b.data_ptr(), ldb,
         b_scales.data_ptr(), None if bias is None else bias.data_ptr(), c.data_ptr(), code, ldc)
    return c


def int8_gemm_gated(a, a_scales, b, b_scales, act=ACT_SILU, out_dtype=torch.bfloat16, h=None, stream=None):
    """h[M][F] = act(g) * u with g and u the int8_gemm products of a [M][K] and the stacked gate and up weights
    b [2F][K]."""
    lda, ldb = _ints(a, "a"), _ints(b, "b")
    (m, k), n2, dev = a.shape, b.shape[0], a.device
    if b.shape[1] != k:
        raise ValueError("a and b disagree on K")
    if n2 % 2:
        raise ValueError("b must hold as many gate rows as up rows")
    _expect(b, "b", torch.int8, (n2, k), dev)
    _expect(a_scales, "a_scales", torch.float32, (m,), dev, dense=True)
    _expect(b_scales, "b_scales", torch.float32, (n2,), dev, dense=True)
    h, code, ldh = _out(h, "h", out_dtype, m, n2 // 2, dev)
    _run(lib.int8_gemm_gated, dev, stream, act, m, n2 // 2, k, a.data_ptr(), lda, a_scales.data_ptr(),
         b.data_ptr(), ldb, b_scales.data_ptr(), h.data_ptr(), code, ldh)
    return h
