"""Binding of the operators in front of the projections (include/fp8q_front.h).

    fp8_rmsnorm(x, weight, residual, transposed)     -> (q, scales[, q_t, scales_t][, h][, rstd][, y])
    int8_rmsnorm(x, weight, residual)                -> (q, scales[, h][, rstd][, y])
    rmsnorm_backward(dy, h, weight, rstd, dh)        -> (dx, dw)
    moe_route(logits, k, valid, renormalize)         -> (weights, experts, counts, loss, slope)
    moe_route_backward(logits, experts, slope, ...)  -> dlogits
    fp8_moe_dispatch(experts, q, scales, E)          -> (a, a_scales, group_of_mtile, row_of_slot, token_of_row)
Argument marshalling only, like the package's other entry points.  Workspaces
are allocated for each call, on the stream it goes to.  Outputs that the
binding allocates have rows a multiple of 16 bytes apart, so a tensor whose
last dimension is no such multiple comes back as a view of wider rows.
"""

import ctypes

import torch

from . import ERR_NULL, MAXABS, _cdiv, _check, _codes, _expect, _i64, _int, _outputs_on, _ptr, _rowmajor, lib
from .ffn import _CODE, _call, _done, _f32, _i8, _ld, _native, _out

_f = ctypes.c_float

# (name, argtypes) for every entry point of include/fp8q_front.h that returns a status
SIGNATURES = {
    "fp8_rmsnorm": [_ptr, _i64, _ptr, _i64, _int, _i64, _i64, _ptr, _int, _f, _int, _ptr, _i64, _ptr, _ptr, _i64, _ptr,
                    _i64, _ptr, _ptr, _i64, _ptr, _ptr],
    "int8_rmsnorm": [_ptr, _i64, _ptr, _i64, _int, _i64, _i64, _ptr, _int, _f, _ptr, _i64, _ptr, _ptr, _i64, _ptr, _i64,
                     _ptr, _ptr],
    "rmsnorm_backward": [_ptr, _i64, _ptr, _i64, _int, _i64, _i64, _ptr, _int, _ptr, _ptr, _i64, _ptr, _i64, _ptr, _int,
                         _ptr, _ptr],
    "moe_route": [_ptr, _i64, _int, _i64, _i64, _i64, _ptr, _int, _ptr, _ptr, _ptr, _ptr, _ptr, _ptr, _ptr],
    "moe_route_backward": [_ptr, _i64, _int, _i64, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _int, _ptr, _i64, _ptr],
    "fp8_moe_dispatch": [_ptr, _i64, _i64, _i64, _ptr, _i64, _ptr, _i64, _i64, _ptr, _i64, _ptr, _ptr, _ptr, _ptr, _ptr,
                         _ptr],
}

# sizes in bytes or rows; -1 where there are no such sizes
SIZES = {
    "fp8q_rmsnorm_backward_workspace": [_i64, _i64],
    "fp8q_moe_route_workspace": [_i64, _i64],
    "fp8q_moe_dispatch_workspace": [_i64, _i64, _i64],
    "fp8q_moe_max_rows": [_i64, _i64, _i64],
}

for _name, _argtypes in {**SIGNATURES, **SIZES}.items():
    getattr(lib, _name).argtypes = _argtypes
    getattr(lib, _name).restype = _i64 if _name in SIZES else ctypes.c_int

_i32 = torch.int32

# The usual call (new outputs, current device and stream) is made by csrc/front/binding.cpp in one step; it answers None
# for anything else, and an int where the C ABI refuses.  What follows it here takes every call, and says what is wrong
# with one.  (A module that was built from csrc/ffn/ alone has no such functions.)
_native = _native if hasattr(_native, "fp8_rmsnorm") else None


def _code(t, name):
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _weight(w, d, dev):
    if w.dtype not in _CODE:
        raise TypeError(f"weight must be bfloat16 or float32, got {w.dtype}")
    _expect(w, "weight", w.dtype, (d,), dev, dense=True)
    return _CODE[w.dtype]


def _given(t, name, dtype, shape, dev):
    """Pointer of an optional packed array."""
    if t is None:
        return None
    return _expect(t, name, dtype, shape, dev, dense=True).data_ptr()


def _packed(t, name, dtype, shape, dev):
    """The caller's packed array, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return _expect(t, name, dtype, shape, dev, dense=True)


def _scratch(size, dev):
    """Workspace of the bytes that one of SIZES answered; sizes that there are none of are the entry point's to refuse."""
    return torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None


def _at(t):
    return None if t is None else t.data_ptr()


def _norm_inputs(x, weight, residual, h):
    _rowmajor(x, "x")
    (m, d), dev, code = x.shape, x.device, _code(x, "x")
    w_code = _weight(weight, d, dev)
    if residual is not None:
        _expect(residual, "residual", x.dtype, (m, d), dev)
    elif h is not None:
        raise ValueError("h is the sum with a residual: there is none")
    return m, d, dev, code, w_code


def _norm_outputs(x, residual, h, rstd, y, save_rstd, save_y):
    """h, rstd and y as the call leaves them (None: not asked for) and their leading dimensions."""
    (m, d), dev = x.shape, x.device
    ld_h = ld_y = 0
    if residual is not None:
        h, _, ld_h = _out(h, "h", x.dtype, m, d, dev)
        _same_type(h, "h", x)
    if rstd is not None or save_rstd:
        rstd = _packed(rstd, "rstd", _f32, (m,), dev)
    if y is not None or save_y:
        y, _, ld_y = _out(y, "y", x.dtype, m, d, dev)
        _same_type(y, "y", x)
    return h, ld_h, rstd, y, ld_y


def _same_type(t, name, x):
    if t.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype} like x, got {t.dtype}")


def fp8_rmsnorm(x, weight, residual=None, eps=1e-6, mode=MAXABS, transposed=False, save_rstd=False, save_y=False,
                h=None, rstd=None, y=None, q=None, scales=None, q_t=None, scales_t=None, stream=None):
    """Root-mean-square norm of h = x (+ residual, rounded to x's type) times `weight`, in FP8: q [M][D] in 1x128 tiles,
    scales [D/128][M].  Then, as far as asked for: with transposed=True also q_t [D][Mp] and scales_t [Mp/128][D]
    (128x1 tiles, Wgrad's operand), Mp being M rounded up to whole 128-row tiles, which q and scales then have too, the
    rows past M zero; h where there is a residual; rstd [M] with save_rstd=True, for rmsnorm_backward; y itself, in
    x's type, with save_y=True.  Giving an output's tensor asks for it."""
    if _native and stream is None and h is None and rstd is None and y is None and q is None and scales is None and \
            q_t is None and scales_t is None:
        r = _native.fp8_rmsnorm(x, weight, residual, eps, mode, transposed, save_rstd, save_y)
        if r is not None:
            return _done(r)
    m, d, dev, code, w_code = _norm_inputs(x, weight, residual, h)
    if not transposed and (q_t is not None or scales_t is not None):
        raise ValueError("q_t / scales_t are the transposed copy: pass transposed=True")
    mq = m + -m % 128 if transposed else m
    keep_rstd = save_rstd or rstd is not None
    with _outputs_on(stream, dev, q, scales, *((q_t, scales_t, rstd) if transposed else ()),
                     *((h,) if residual is not None else ()), *((rstd,) if save_rstd else ()),
                     *((y,) if save_y else ())):
        h, ld_h, rstd, y, ld_y = _norm_outputs(x, residual, h, rstd, y, save_rstd or transposed, save_y)
        if q is None:
            q = torch.empty((mq, d), dtype=torch.uint8, device=dev)
        scales = _packed(scales, "scales", _f32, (_cdiv(d, 128), mq), dev)
        if transposed:
            if q_t is None:
                q_t = torch.empty((d, mq), dtype=torch.uint8, device=dev)
            scales_t = _packed(scales_t, "scales_t", _f32, (_cdiv(mq, 128), d), dev)
    q = _expect(_codes(q), "q", torch.uint8, (mq, d), dev)
    ld_qt = 0
    if transposed:
        q_t = _expect(_codes(q_t), "q_t", torch.uint8, (d, mq), dev)
        ld_qt = _ld(q_t)
    _call(lib.fp8_rmsnorm, dev, stream, x.data_ptr(), _ld(x), _at(residual), 0 if residual is None else _ld(residual),
          code, m, d, weight.data_ptr(), w_code, eps, mode, _at(h), ld_h, _at(rstd), _at(y), ld_y, q.data_ptr(), _ld(q),
          scales.data_ptr(), _at(q_t), ld_qt, _at(scales_t))
    out = (q, scales, q_t, scales_t) if transposed else (q, scales)
    if h is not None:
        out += (h,)
    if keep_rstd:
        out += (rstd,)
    return out if y is None else out + (y,)


def int8_rmsnorm(x, weight, residual=None, eps=1e-6, save_rstd=False, save_y=False, h=None, rstd=None, y=None, q=None,
                 scales=None, stream=None):
    """The norm of fp8_rmsnorm in 8-bit integers with one scale for each row: q int8 [M][D], scales [M], and h, rstd and
    y as far as asked for."""
    if _native and stream is None and h is None and rstd is None and y is None and q is None and scales is None:
        r = _native.int8_rmsnorm(x, weight, residual, eps, save_rstd, save_y)
        if r is not None:
            return _done(r)
    m, d, dev, code, w_code = _norm_inputs(x, weight, residual, h)
    with _outputs_on(stream, dev, q, scales, *((h,) if residual is not None else ()), *((rstd,) if save_rstd else ()),
                     *((y,) if save_y else ())):
        h, ld_h, rstd, y, ld_y = _norm_outputs(x, residual, h, rstd, y, save_rstd, save_y)
        if q is None:
            ld = max(d + -d % 16, 16)              # the last row's bytes up to 16 exist too, as int8_gemm reads them
            q = torch.empty(m, ld, dtype=_i8, device=dev)
            if ld != d:
                q = q.as_strided((m, d), (ld, 1))
        else:
            _expect(q, "q", _i8, (m, d), dev)
        scales = _packed(scales, "scales", _f32, (m,), dev)
    _call(lib.int8_rmsnorm, dev, stream, x.data_ptr(), _ld(x), _at(residual), 0 if residual is None else _ld(residual),
          code, m, d, weight.data_ptr(), w_code, eps, _at(h), ld_h, _at(rstd), _at(y), ld_y, q.data_ptr(), _ld(q),
          scales.data_ptr())
    return (q, scales) + tuple(t for t in (h, rstd, y) if t is not None)


def rmsnorm_backward(dy, h, weight, rstd, dh=None, dx=None, dw=None, accumulate=False, stream=None):
    """Gradient of the norm y = h rstd weight: dx [M][D] of h (of x and of the residual alike), with dh, the gradient that
    reaches h past the norm, added, and dw FP32 [D] of the weight, added to dw with accumulate=True."""
    if _native and stream is None and dx is None and dw is None and not accumulate:
        r = _native.rmsnorm_backward(dy, h, weight, rstd, dh)
        if r is not None:
            return _done(r)
    _rowmajor(dy, "dy")
    (m, d), dev, code = dy.shape, dy.device, _code(dy, "dy")
    _expect(h, "h", dy.dtype, (m, d), dev)
    w_code = _weight(weight, d, dev)
    _expect(rstd, "rstd", _f32, (m,), dev, dense=True)
    if dh is not None:
        _expect(dh, "dh", dy.dtype, (m, d), dev)
    if accumulate and dw is None:
        raise ValueError("accumulate=True adds to dw: pass it")
    with _outputs_on(stream, dev, None):
        dx, _, ld_dx = _out(dx, "dx", dy.dtype, m, d, dev)
        dw = _packed(dw, "dw", _f32, (d,), dev)
        work = _scratch(lib.fp8q_rmsnorm_backward_workspace(m, d), dev)
    if dx.dtype != dy.dtype:
        raise TypeError(f"dx must be {dy.dtype} like dy, got {dx.dtype}")
    _call(lib.rmsnorm_backward, dev, stream, dy.data_ptr(), _ld(dy), h.data_ptr(), _ld(h), code, m, d, weight.data_ptr(),
          w_code, rstd.data_ptr(), _at(dh), 0 if dh is None else _ld(dh), dx.data_ptr(), ld_dx, dw.data_ptr(),
          1 if accumulate else 0, _at(work))
    return dx, dw


def moe_route(logits, k, valid=None, renormalize=False, weights=None, experts=None, counts=None, loss=None, slope=None,
              stream=None):
    """The k experts of each token: weights FP32 [T][k], their softmax probabilities (over their sum with
    renormalize=True), experts int32 [T][k] in descending order, counts int32 [E], loss FP32 [1], the balance loss
    E sum_e f_e P_e, and slope FP32 [E], its gradient by each token's probabilities.  valid (bool or uint8 [T]) says
    which tokens count; the others have experts -1.  A logit of minus infinity is never chosen."""
    if _native and stream is None and weights is None and experts is None and counts is None and loss is None and \
            slope is None:
        r = _native.moe_route(logits, k, valid, renormalize)
        if r is not None:
            return _done(r)
    _rowmajor(logits, "logits")
    (t, e), dev, code, k = logits.shape, logits.device, _code(logits, "logits"), int(k)
    if valid is not None:
        _expect(valid, "valid", torch.bool if valid.dtype == torch.bool else torch.uint8, (t,), dev, dense=True)
    # sizes are the entry point's to refuse, before memory is asked for: it looks at pointers behind them
    status = lib.moe_route(None, _ld(logits), code, t, e, k, None, 0, None, None, None, None, None, None, None)
    if status != ERR_NULL:
        _check(status)
    with _outputs_on(stream, dev, None):
        weights = _packed(weights, "weights", _f32, (t, k), dev)
        experts = _packed(experts, "experts", _i32, (t, k), dev)
        counts = _packed(counts, "counts", _i32, (e,), dev)
        loss = _packed(loss, "loss", _f32, (1,), dev)
        slope = _packed(slope, "slope", _f32, (e,), dev)
        work = _scratch(lib.fp8q_moe_route_workspace(t, e), dev)
    _call(lib.moe_route, dev, stream, logits.data_ptr(), _ld(logits), code, t, e, k, _at(valid), 1 if renormalize else 0,
          weights.data_ptr(), experts.data_ptr(), counts.data_ptr(), loss.data_ptr(), slope.data_ptr(), _at(work))
    return weights, experts, counts, loss, slope


def moe_route_backward(logits, experts, slope=None, dweights=None, dloss=None, renormalize=False, dlogits=None,
                       stream=None):
    """Gradient of moe_route's weights and loss with respect to the logits, in their type, from dweights FP32 [T][k]
    and dloss FP32 [1] (either may be None: zero); experts and slope as moe_route left them."""
    if _native and stream is None and dlogits is None:
        r = _native.moe_route_backward(logits, experts, slope, dweights, dloss, renormalize)
        if r is not None:
            return _done(r)
    _rowmajor(logits, "logits")
    (t, e), dev, code = logits.shape, logits.device, _code(logits, "logits")
    if experts.dim() != 2:
        raise ValueError("experts must be a [T][k] tensor")
    k = experts.shape[1]
    _expect(experts, "experts", _i32, (t, k), dev, dense=True)
    if dloss is not None and slope is None:
        raise ValueError("dloss goes by slope: pass it")
    slope_ptr, dw_ptr = _given(slope, "slope", _f32, (e,), dev), _given(dweights, "dweights", _f32, (t, k), dev)
    dl_ptr = _given(dloss, "dloss", _f32, (1,), dev)
    with _outputs_on(stream, dev, dlogits):
        dlogits, _, ld = _out(dlogits, "dlogits", logits.dtype, t, e, dev)
    if dlogits.dtype != logits.dtype:
        raise TypeError(f"dlogits must be {logits.dtype} like logits, got {dlogits.dtype}")
    _call(lib.moe_route_backward, dev, stream, logits.data_ptr(), _ld(logits), code, t, e, k, experts.data_ptr(),
          slope_ptr, dw_ptr, dl_ptr, 1 if renormalize else 0, dlogits.data_ptr(), ld)
    return dlogits


def moe_max_rows(tokens, k, num_experts):
    """Rows of whole 128-row tiles that `tokens` tokens of k experts each take at most."""
    rows = lib.fp8q_moe_max_rows(tokens, k, num_experts)
    if rows < 0:
        raise ValueError(f"no such sizes: {tokens} tokens of {k} of {num_experts} experts")
    return rows


def fp8_moe_dispatch(experts, q, scales, num_experts, a=None, a_scales=None, group_of_mtile=None, row_of_slot=None,
                     token_of_row=None, stream=None):
    """Operand and tile map of fp8_gemm_blockscaled_grouped: the rows q [T][D] (1x128 tiles, scales [D/128][T]) of each
    token's experts [T][k], in the order of the experts and each expert's rows padded with zeros to whole 128-row
    tiles.  a [M][D], a_scales [D/128][M], group_of_mtile int32 [M/128] (-1: tile not in use, whose rows and scales are
    left as they are), row_of_slot int32 [T][k] (-1 for experts outside the range), token_of_row int32 [M] (-1: none).
    M is moe_max_rows(T, k, E), or what the first given one of a, a_scales, group_of_mtile and token_of_row has."""
    if _native and stream is None and group_of_mtile is None and row_of_slot is None and token_of_row is None:
        r = _native.fp8_moe_dispatch(experts, q, scales, num_experts, a, a_scales)
        if r is not None:
            return _done(r)
    q = _codes(_rowmajor(q, "q"))
    (t, d), dev, e = q.shape, q.device, int(num_experts)
    if experts.dim() != 2:
        raise ValueError("experts must be a [T][k] tensor")
    k = experts.shape[1]
    _expect(experts, "experts", _i32, (t, k), dev, dense=True)
    g = _cdiv(d, 128)
    _expect(scales, "scales", _f32, (g, t), dev, dense=True)
    if a is not None:
        rows = a.shape[0]
    elif a_scales is not None:
        rows = a_scales.shape[-1]
    elif group_of_mtile is not None:
        rows = 128 * group_of_mtile.shape[0]
    elif token_of_row is not None:
        rows = token_of_row.shape[0]
    else:
        rows = moe_max_rows(t, k, e)
    with _outputs_on(stream, dev, None):
        if a is None:
            a = torch.empty((rows, d), dtype=torch.uint8, device=dev)
        a_scales = _packed(a_scales, "a_scales", _f32, (g, rows), dev)
        group_of_mtile = _packed(group_of_mtile, "group_of_mtile", _i32, (_cdiv(rows, 128),), dev)
        row_of_slot = _packed(row_of_slot, "row_of_slot", _i32, (t, k), dev)
        token_of_row = _packed(token_of_row, "token_of_row", _i32, (rows,), dev)
        work = _scratch(lib.fp8q_moe_dispatch_workspace(t, k, e), dev)
    a = _expect(_codes(a), "a", torch.uint8, (rows, d), dev)
    _call(lib.fp8_moe_dispatch, dev, stream, experts.data_ptr(), t, k, e, q.data_ptr(), _ld(q), scales.data_ptr(), d, rows,
          a.data_ptr(), _ld(a), a_scales.data_ptr(), group_of_mtile.data_ptr(), row_of_slot.data_ptr(),
          token_of_row.data_ptr(), _at(work))
    return a, a_scales, group_of_mtile, row_of_slot, token_of_row
