"""fp8_rmsnorm, int8_rmsnorm and rmsnorm_backward on the GPU against the 64-bit definitions of oracle/front.py.

Forward: h is exact (one FP32 sum, rounded), rstd has a tolerance, and everything after it is stated FP32 operations on
h, rstd and weight, so y, codes and scales follow bit for bit from the rstd that the GPU returns.

Tolerances, with u = 2^-24:
  * a row's sum adds at most 32 products per thread one after the other (fused: one rounding each), 6 lane steps and 16
    waves: 54 roundings, a relative 54 u of a sum of squares; times 1/D (2 u), plus eps (1 u), halved by the root, which
    and the quotient are one rounding each: 31 u for rstd;
  * gradient: xhat = h rstd, z = dy xhat and g = dy w are one rounding each; the mean of z w has 54 roundings, z's two and
    the one of 1/D: 60 u of mean |g xhat|; dx = rstd (g - xhat c) + dh with a fused difference has 4 more;
  * dw: R rows one after the other, then up to 32 parts and 16 partial sums, z's two roundings and up to 16 rows that meet
    in the workgroup, and one to accumulate;
  * BF16 outputs: half a step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

from oracle import ffn as of, front as orf, quant as oq
from tests.helpers import assert_bytes_equal, dev, host, require_gpu
from workloads import add_outliers, bf16_bits_as_f32, normal_f32, to_bf16_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF, I8 = torch.float32, torch.bfloat16, torch.int8
EPS = 1e-6


def _round(x, dtype):
    return bf16_bits_as_f32(to_bf16_bits(x)) if dtype == BF else np.asarray(x, np.float32)


def _values(rng, shape, sigma, dtype, outliers=0.01):
    return _round(add_outliers(rng, normal_f32(rng, shape, sigma), outliers, 50.0), dtype)


def _up(n, to):
    return -(-n // to) * to


def _place(x, dtype, extra=1):
    """A float32 array as a device view of `dtype` with rows further apart than they are long, NaN in the gaps."""
    rows, cols = x.shape
    per = 16 // torch.empty((), dtype=dtype).element_size()
    buf = torch.full((rows, _up(max(cols, 1), per) + extra * per), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = dev(x).to(dtype)
    return buf[:, :cols]


def _guarded(rows, cols, dtype, fill=-77):
    per = 16 // torch.empty((), dtype=dtype).element_size()
    buf = torch.full((rows + 2, _up(cols, per) + per), fill, dtype=dtype, device="cuda")

    def intact():
        b = buf.clone()
        b[1:rows + 1, :cols] = fill
        assert bool((b == fill).all()), "written outside the output"
    return buf[1:rows + 1, :cols], intact


def _case(m, d, dtype, wdtype, residual, seed=None):
    rng = np.random.default_rng(m * 100003 + d if seed is None else seed)
    x = _values(rng, (m, d), 1.0, dtype)
    r = _values(rng, (m, d), 2.0, dtype, 0.0) if residual else None
    if m > 2:
        x[1] = 0.0                                        # a row of zeros
        x[2] *= np.float32(2.0 ** -60)                    # a row that eps outweighs
        if residual:
            r[1] = 0.0
            r[2] = 0.0
    w = _round(1.0 + normal_f32(rng, (d,), 0.3), wdtype)
    if d > 5:
        w[5] = 0.0
        w[3] = -w[3]
    h = _round(x + r, dtype) if residual else x           # one FP32 sum, rounded
    return x, r, w, h


def _check_forward(h, w, dtype, got_h, got_rstd, got_y, residual):
    """h exactly, rstd within its tolerance; returns the FP32 y that follows from them."""
    if residual:
        assert_bytes_equal(host(got_h.float()), h, "h")
    rstd = host(got_rstd)
    ref = orf.rstd(h, EPS)
    assert np.all(np.abs(rstd - ref) <= 31 * U * ref), np.max(np.abs(rstd / ref - 1)) / U
    y = ((h * rstd[:, None]).astype(np.float32) * w[None, :]).astype(np.float32)
    if got_y is not None:
        assert_bytes_equal(host(got_y.float()), _round(y, dtype), "y")
    return y


WIDTHS = [128, 256, 384, 512, 640, 1024, 1152, 2048, 2176, 4096, 4224, 8192, 8320, 16384, 16512, 32768]


@pytest.mark.parametrize("dtype, wdtype", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("m, d", [(1, 128), (3, 7168), (130, 384), (5, 2048)] + [(4, d) for d in WIDTHS])
def test_fp8_rmsnorm(m, d, dtype, wdtype):
    fp8q = require_gpu()
    residual, mode = (m + d // 128) % 3 != 0, (d // 128) % 2
    x, r, w, h = _case(m, d, dtype, wdtype, residual)
    q, q_ok = _guarded(m, d, torch.uint8, 0x55)
    y, y_ok = _guarded(m, d, dtype)
    hh, h_ok = _guarded(m, d, dtype)
    kw = dict(residual=_place(r, dtype, 2), h=hh) if residual else {}
    out = fp8q.fp8_rmsnorm(_place(x, dtype), dev(w).to(wdtype), eps=EPS, mode=mode, save_rstd=True, y=y, q=q, **kw)
    assert len(out) == (5 if residual else 4)
    y32 = _check_forward(h, w, dtype, hh, out[-2], y, residual)
    want_q, want_s = oq.quant_1x128(y32, "pow2" if mode else "maxabs")
    assert_bytes_equal(host(out[1]), want_s, "scales")
    assert_bytes_equal(host(q), want_q, "codes")
    for ok in (q_ok, y_ok, h_ok):
        ok()
    again = fp8q.fp8_rmsnorm(_place(x, dtype), dev(w).to(wdtype), eps=EPS, mode=mode,
                             **({"residual": _place(r, dtype)} if residual else {}))
    assert len(again) == (3 if residual else 2)           # outputs of the binding
    assert torch.equal(again[0], q) and torch.equal(again[1], out[1]) and (not residual or torch.equal(again[2], hh))


@pytest.mark.parametrize("dtype, wdtype", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("m, d", [(1, 128), (127, 256), (128, 128), (129, 384), (300, 1280), (5, 7168), (256, 2048)])
@pytest.mark.parametrize("residual", [False, True])
def test_fp8_rmsnorm_both_tilings(m, d, dtype, wdtype, residual):
    fp8q = require_gpu()
    mode, mp = (m + d // 128) % 2, _up(m, 128)
    x, r, w, h = _case(m, d, dtype, wdtype, residual)
    q, q_ok = _guarded(mp, d, torch.uint8, 0x55)
    qt, qt_ok = _guarded(d, mp, torch.uint8, 0x55)
    y, y_ok = _guarded(m, d, dtype)
    kw = dict(residual=_place(r, dtype)) if residual else {}
    out = fp8q.fp8_rmsnorm(_place(x, dtype), dev(w).to(wdtype), eps=EPS, mode=mode, transposed=True, save_rstd=True, q=q,
                           q_t=qt, y=y, **kw)
    y32 = np.zeros((mp, d), np.float32)
    y32[:m] = _check_forward(h, w, dtype, out[4], out[-2], y, residual)
    name = "pow2" if mode else "maxabs"
    want = oq.quant_1x128(y32, name) + oq.quant_128x1(y32, name)
    for got, ref, what in zip(out, want, ("1x128 codes", "1x128 scales", "128x1 codes", "128x1 scales")):
        assert_bytes_equal(host(got), ref, what)
    for ok in (q_ok, qt_ok, y_ok):
        ok()
    # what the single tiling gives is what both give
    one = fp8q.fp8_rmsnorm(_place(x, dtype), dev(w).to(wdtype), eps=EPS, mode=mode, **kw)
    assert torch.equal(one[0], out[0][:m]) and torch.equal(one[1], out[1][:, :m])
    # without rstd and h asked for
    two = fp8q.fp8_rmsnorm(_place(x, dtype), dev(w).to(wdtype), eps=EPS, mode=mode, transposed=True, **kw)
    assert len(two) == (5 if residual else 4) and all(torch.equal(a, b) for a, b in zip(two, out[:4]))


@pytest.mark.parametrize("dtype, wdtype", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("m, d", [(1, 1), (3, 7), (5, 9), (2, 129), (130, 333), (4, 1023), (3, 2047), (2, 4097), (5, 7168), (1, 8191),
                                  (2, 16383), (1, 32767), (4, 511), (6, 513)])
def test_int8_rmsnorm(m, d, dtype, wdtype):
    fp8q = require_gpu()
    residual = (m + d) % 2 == 0
    x, r, w, h = _case(m, d, dtype, wdtype, residual)
    q, q_ok = _guarded(m, d, I8)
    y, y_ok = _guarded(m, d, dtype)
    hh, h_ok = _guarded(m, d, dtype)
    kw = dict(residual=_place(r, dtype), h=hh) if residual else {}
    out = fp8q.int8_rmsnorm(_place(x, dtype), dev(w).to(wdtype), eps=EPS, save_rstd=True, y=y, q=q, **kw)
    y32 = _check_forward(h, w, dtype, hh, out[-2], y, residual)
    want_q, want_s = of.quant_int8_rows(y32)
    assert_bytes_equal(host(out[1]), want_s, "scales")
    assert_bytes_equal(host(q), want_q, "codes")
    for ok in (q_ok, y_ok, h_ok):
        ok()
    again = fp8q.int8_rmsnorm(_place(x, dtype), dev(w).to(wdtype), eps=EPS, **kw)
    assert torch.equal(again[0], q) and torch.equal(again[1], out[1])


def test_norm_of_extreme_rows():
    """Rows of zeros (scales of zeros, rstd of eps), of the smallest numbers, and of 1e17, whose squares nearly overflow."""
    fp8q = require_gpu()
    x = np.zeros((4, 256), np.float32)
    x[1] = 2.0 ** -149
    x[2] = 1e17
    x[3, 0] = 3e18
    w = np.ones(256, np.float32)
    q, s, rstd, y = fp8q.fp8_rmsnorm(dev(x), dev(w), eps=1e-30, save_rstd=True, save_y=True)
    _check = orf.norm(x, w, 1e-30)
    assert bool(torch.isfinite(y).all()) and np.all(np.abs(host(y) - _check) <= 33 * U * np.abs(_check) + 2.0 ** -126)
    assert not q[:1].any() and bool((s[:, 0] == 2.0 ** -126).all())
    # the limit on rows for which the squares' mean is what counts: eps alone
    assert abs(float(rstd[0]) * 1e-15 - 1.0) <= 4 * U


def test_norm_empty():
    fp8q = require_gpu()
    e = torch.empty((0, 256), device="cuda")
    w = torch.ones(256, device="cuda")
    q, s, qt, st, rstd = fp8q.fp8_rmsnorm(e, w, transposed=True, save_rstd=True)
    assert q.shape == (0, 256) and s.shape == (2, 0) and qt.shape == (256, 0) and st.shape == (0, 256) and rstd.shape == (0,)
    q, s = fp8q.int8_rmsnorm(e, w)
    assert q.shape == (0, 256) and s.shape == (0,)
    n = torch.empty((3, 0), device="cuda")
    q, s, rstd = fp8q.int8_rmsnorm(n, w[:0], eps=0.25, save_rstd=True)
    assert q.shape == (3, 0) and bool((s == 2.0 ** -126).all()) and bool((rstd == 2.0).all())
    dw = torch.full((256,), 3.0, device="cuda")
    fp8q.rmsnorm_backward(e, e, w, w[:0], dw=dw, accumulate=True)
    assert bool((dw == 3.0).all())
    dx, dw = fp8q.rmsnorm_backward(e, e, w, w[:0])
    assert dx.shape == (0, 256) and not dw.any()


# ---------------------------------------------------------------------------
# rmsnorm_backward
# ---------------------------------------------------------------------------
BWD = [(1, 1), (3, 7), (2, 129), (5000, 250), (130, 333), (9, 512), (70, 1023), (33, 2047), (20, 4097), (700, 2048), (5, 7168), (3, 8191),
       (2, 16383), (300, 8200), (2, 32767), (1, 32768), (2100, 64), (4500, 520), (513, 1500), (1030, 1032)]


@pytest.mark.parametrize("dtype, wdtype", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("m, d", BWD)
def test_rmsnorm_backward(m, d, dtype, wdtype):
    fp8q = require_gpu()
    rng = np.random.default_rng(m * 7 + d)
    _, _, w, h = _case(m, d, dtype, wdtype, False)
    dy = _values(rng, (m, d), 1e-3, dtype)
    dh = _values(rng, (m, d), 1e-3, dtype) if (m + d) % 3 else None
    r = orf.rstd(h, EPS).astype(np.float32)
    dx, dx_ok = _guarded(m, d, dtype)
    dw = torch.full((d,), float("nan"), device="cuda")
    fp8q.rmsnorm_backward(_place(dy, dtype, 2), _place(h, dtype), dev(w).to(wdtype), dev(r),
                          dh=None if dh is None else _place(dh, dtype), dx=dx, dw=dw)
    dx_ok()
    ref_x, ref_w = orf.norm_backward(dy, h, w, r, dh)
    xhat = np.abs(h.astype(np.float64) * r[:, None])
    g = np.abs(dy.astype(np.float64) * w)
    mean = (g * xhat).mean(axis=1, keepdims=True)
    tol = r[:, None].astype(np.float64) * (4 * g + (4 + 60) * xhat * mean) * U + 2 * U * np.abs(ref_x) + 2.0 ** -120
    if dh is not None:
        tol += U * np.abs(dh)
    tol += np.abs(ref_x) * 2.0 ** -8 if dtype == BF else 0.0
    err = np.abs(dx.double().cpu().numpy() - ref_x)
    assert np.all(err <= tol), np.max(err / tol)
    # a workgroup's turns: one row each of at least 256 of them; then parts, their sums, and up to 16 rows that meet
    steps = -(-m // 256) + 32 + 16 + 2 + 16 + 1
    scale = (np.abs(dy.astype(np.float64)) * xhat).sum(axis=0)
    err = np.abs(dw.double().cpu().numpy() - ref_w)
    assert np.all(err <= steps * U * scale + 2.0 ** -120), np.max(err / (steps * U * scale + 2.0 ** -120))
    # accumulated: the same sum added to what was there
    start = torch.randn(d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    acc = start.clone()
    dx2, same = fp8q.rmsnorm_backward(_place(dy, dtype), _place(h, dtype), dev(w).to(wdtype), dev(r),
                                      dh=None if dh is None else _place(dh, dtype), dw=acc, accumulate=True)
    assert same is acc and torch.equal(acc, start + dw) and torch.equal(dx2, dx)


def test_rmsnorm_backward_against_differences():
    """The GPU's gradient against central differences of the 64-bit forward pass (step 1e-6: under 1e-8 off), in FP32."""
    fp8q = require_gpu()
    rng = np.random.default_rng(8)
    m, d, eps, step = 3, 24, 0.05, 1e-6
    h, w = normal_f32(rng, (m, d), 1.0), 1.0 + normal_f32(rng, (d,), 0.3)
    dy, dh = normal_f32(rng, (m, d), 1.0), normal_f32(rng, (m, d), 1.0)
    rstd = fp8q.int8_rmsnorm(dev(h), dev(w), eps=eps, save_rstd=True)[2]
    dx, dw = fp8q.rmsnorm_backward(dev(dy), dev(h), dev(w), rstd, dh=dev(dh))
    h, w = h.astype(np.float64), w.astype(np.float64)
    f = lambda h_, w_: float((orf.norm(h_, w_, eps) * dy).sum() + (h_ * dh).sum())      # noqa: E731
    for i in np.ndindex(m, d):
        e = np.zeros((m, d))
        e[i] = step
        num = (f(h + e, w) - f(h - e, w)) / (2 * step)
        assert abs(float(dx[i]) - num) <= 1e-8 + 200 * U * 10      # terms of order 10 at most, 100 roundings and rstd's
    for i in range(d):
        e = np.zeros(d)
        e[i] = step
        assert abs(float(dw[i]) - (f(h, w + e) - f(h, w - e)) / (2 * step)) <= 1e-8 + 200 * U * 10


def test_norm_refusals():
    fp8q = require_gpu()
    f = lambda *s: torch.ones(s, device="cuda")                          # noqa: E731
    x, w = f(4, 256), f(256)
    with pytest.raises(ValueError, match="residual has shape"):
        fp8q.fp8_rmsnorm(x, w, residual=f(4, 128))
    with pytest.raises(TypeError, match="residual must be"):
        fp8q.fp8_rmsnorm(x, w, residual=x.to(BF))
    with pytest.raises(ValueError, match="weight has shape"):
        fp8q.int8_rmsnorm(x, f(255))
    with pytest.raises(TypeError, match="weight must be"):
        fp8q.int8_rmsnorm(x, w.half())
    with pytest.raises(TypeError, match="x must be"):
        fp8q.int8_rmsnorm(x.half(), w)
    with pytest.raises(ValueError, match="h is the sum"):
        fp8q.fp8_rmsnorm(x, w, h=f(4, 256))
    with pytest.raises(ValueError, match="transposed=True"):
        fp8q.fp8_rmsnorm(x, w, q_t=torch.empty((256, 128), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="q has shape"):              # whole 128-row tiles
        fp8q.fp8_rmsnorm(x, w, transposed=True, q=torch.empty((4, 256), dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="y must be"):
        fp8q.fp8_rmsnorm(x, w, y=x.to(BF))
    with pytest.raises(ValueError, match="row-major"):
        fp8q.fp8_rmsnorm(f(256, 4).t(), w)
    for bad, status in ((dict(eps=0.0), fp8q.ERR_ARG), (dict(mode=3), fp8q.ERR_ARG), (dict(residual=x, h=x), fp8q.ERR_ALIAS)):
        with pytest.raises(fp8q.Fp8qError) as e:
            fp8q.fp8_rmsnorm(x, w, **bad)
        assert e.value.status == status
    with pytest.raises(fp8q.Fp8qError) as e:
        fp8q.fp8_rmsnorm(f(4, 208), f(208))
    assert e.value.status == fp8q.ERR_UNSUPPORTED
    with pytest.raises(fp8q.Fp8qError) as e:
        fp8q.int8_rmsnorm(f(1, 32769), f(32769))
    assert e.value.status == fp8q.ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="accumulate=True adds to dw"):
        fp8q.rmsnorm_backward(x, x, w, f(4), accumulate=True)
    with pytest.raises(ValueError, match="rstd has shape"):
        fp8q.rmsnorm_backward(x, x, w, f(5))
    with pytest.raises(TypeError, match="h must be"):
        fp8q.rmsnorm_backward(x, x.to(BF), w, f(4))
    with pytest.raises(TypeError, match="dx must be"):
        fp8q.rmsnorm_backward(x, x, w, f(4), dx=x.to(BF))
    with pytest.raises(fp8q.Fp8qError) as e:
        fp8q.rmsnorm_backward(x, x, w, f(4), dx=x)
    assert e.value.status == fp8q.ERR_ALIAS


@pytest.mark.parametrize("given", [False, True])
def test_rmsnorm_backward_refuses_rows_beyond_the_widest(given):
    """The native call (no output given) and the other one alike."""
    fp8q = require_gpu()
    x, w = torch.ones((2, 32776), device="cuda")[:, :32769], torch.ones(32769, device="cuda")
    with pytest.raises(fp8q.Fp8qError) as e:
        fp8q.rmsnorm_backward(x, x, w, torch.ones(2, device="cuda"), **(dict(dw=torch.zeros_like(w)) if given else {}))
    assert e.value.status == fp8q.ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
# Inputs of more than 96 MB are read past the caches, by kernels of their own
# ---------------------------------------------------------------------------
BIG = 96 << 20


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [128, 256, 512, 1024, 2048, 4096, 7168, 16384, 32768])
def test_norms_of_many_rows_agree_with_those_of_few(d, dtype):
    """Every width's kernels, in all forms: the last rows are what a call on them alone gives."""
    fp8q = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(d)
    es = 2 if dtype == BF else 4
    m = BIG // es // d + 130
    lo = (m - 70) // 128 * 128
    x = torch.randn((m, d), generator=gen, device="cuda", dtype=dtype)
    r = torch.randn((m, d), generator=gen, device="cuda", dtype=dtype)
    w = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype)
    xs, rs = x[lo:].clone(), r[lo:].clone()

    def rows(t):                                          # the tail of an output, whichever way it lies
        return t[lo:] if t.shape[0] == m else t[:, lo:]

    for res in (None, r):
        small = None if res is None else rs
        for call in (lambda a, b: fp8q.fp8_rmsnorm(a, w, residual=b, save_rstd=True, save_y=True),
                     lambda a, b: fp8q.fp8_rmsnorm(a, w, residual=b, mode=fp8q.POW2),
                     lambda a, b: fp8q.int8_rmsnorm(a, w, residual=b)):
            for got, want in zip(call(x, res), call(xs, small)):
                assert torch.equal(rows(got), want)
        got, want = fp8q.fp8_rmsnorm(x, w, residual=res, transposed=True), fp8q.fp8_rmsnorm(xs, w, residual=small, transposed=True)
        assert torch.equal(got[0][lo:], want[0]) and torch.equal(got[1][:, lo:], want[1])
        assert torch.equal(got[2][:, lo:], want[2]) and torch.equal(got[3][lo // 128:], want[3])
    rstd = fp8q.int8_rmsnorm(x, w, save_rstd=True)[2]
    for dh in (None, r):
        dx, dw = fp8q.rmsnorm_backward(r, x, w, rstd, dh=dh)
        dx1, _ = fp8q.rmsnorm_backward(rs, xs, w, rstd[lo:].clone(), dh=None if dh is None else rs)
        assert torch.equal(dx[lo:], dx1)
        ref = torch.zeros(d, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(ref)
        for i in range(0, m, 8192):
            z = r[i:i + 8192].double() * x[i:i + 8192].double() * rstd[i:i + 8192].double()[:, None]
            ref += z.sum(0)
            size += z.abs().sum(0)
        steps = m / 256 + 60                              # at least 256 rows at a time
        assert bool(((dw.double() - ref).abs() <= steps * U * size).all())
