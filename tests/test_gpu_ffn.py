"""Gated feed-forward operators on the GPU against the 64-bit definitions of oracle/ffn.py.

Tolerances, with u = 2^-24 the FP32 unit roundoff:
  * integer product: the sum is exact; converting it, forming sa*sb, multiplying and adding the bias are one rounding
    each, so |y - ref| <= 4 u (|ref - bias| + |ref|);
  * act(g) = g sigma(t): t is formed in three roundings and multiplied by log2(e) (relative error 5 u, so the
    exponent is off by 5 u |t|), exp2 and the reciprocal are good to 2 u, the sum and the products one rounding each:
    relative error <= (16 + 8 |t|) u; a relative error of d in g enters act(g) with the factor |g act'(g) / act(g)|
    <= 1 + 3 |t|.  With d = 4 u (a scaled integer sum): (20 + 20 |t|) u in all, and 2 u more for the product with u;
  * act'(g) = s + g s (1-s) t': each of its two terms to (16 + 8 |t|) u, so the absolute error is that times the sum
    of their magnitudes;
  * results under 2^-100 may be flushed on the way: an absolute 2^-100 (times the operands) is added;
  * BF16 output adds half a unit in the last of 8 bits: 2^-8 of the result covers it with the above;
  * block-scaled FP8 products: relative Frobenius error 2e-4 in FP32 and 1e-3 against the rounded result in BF16, the
    bounds of the plain FP8 GEMMs.
"""

import numpy as np
import pytest
import torch

from oracle import ffn as of, gemm as og, quant as oq
from tests.helpers import assert_bytes_equal, dev, dev_bf16, host, require_gpu
from workloads import add_outliers, bf16_bits_as_f32, normal_f32, random_fp8_operands, to_bf16_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -100
F32, BF, I8 = torch.float32, torch.bfloat16, torch.int8
ACTS = [of.SILU, of.GELU_TANH]


def _up(n, to):
    return -(-n // to) * to


def _t(g, kind):
    g = np.asarray(g, np.float64)
    return g if kind == of.SILU else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _near(got, ref, tol, dtype):
    got = _f64(got) if torch.is_tensor(got) else got
    tol = np.broadcast_to(tol, ref.shape) + (np.abs(ref) * 2.0 ** -8 if dtype == BF else 0.0)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(x[0] for x in np.nonzero(bad))
        raise AssertionError(f"{bad.sum()} of {bad.size} off, first at {i}: got {got[i]!r} want {ref[i]!r} +- {tol[i]!r}")


def _padded(x, fill, ld=None, offset=0):
    """x (numpy int8 [rows][cols]) as a device view with rows ld bytes apart, the gaps holding `fill`."""
    rows, cols = x.shape
    ld = ld or _up(max(cols, 1), 16)
    buf = torch.full((rows + offset, ld), fill, dtype=I8, device="cuda")
    buf[offset:, :cols] = dev(x)
    return buf[offset:, :cols]


def _guarded(rows, cols, dtype):
    """A row-strided output view inside a larger buffer of sentinels, and a check that nothing around it changed."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = _up(cols, per) + per
    buf = torch.full((rows + 2, ld), -77, dtype=dtype, device="cuda")

    def intact():
        b = buf.clone()
        b[1:rows + 1, :cols] = -77
        assert bool((b == -77).all()), "written outside the output"
    return buf[1:rows + 1, :cols], intact


# ---------------------------------------------------------------------------
# int8_quant_rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, cols", [(1, 1), (1, 7), (3, 8), (2, 15), (5, 64), (4, 129), (33, 511), (2, 2048),
                                        (7, 2049), (3, 7168), (2, 16385), (1, 40007)])
def test_int8_quant_rows(rows, cols, dtype):
    fp8q = require_gpu()
    rng = np.random.default_rng(rows * 1000 + cols)
    x = add_outliers(rng, normal_f32(rng, (rows, cols), 1.0), 0.01, 50.0)
    x = bf16_bits_as_f32(to_bf16_bits(x)) if dtype == BF else x
    if rows > 1:
        x[0] = 0.0                                        # a row of zeros keeps a normal scale
        x[1] *= np.float32(2.0 ** -120)                   # small rows: the reciprocal of the scale is large
        x = bf16_bits_as_f32(to_bf16_bits(x)) if dtype == BF else x
    per = 16 // (2 if dtype == BF else 4)
    buf = torch.full((rows, _up(cols, per) + per), 3e38, dtype=dtype, device="cuda")    # the gaps are larger than any value
    buf[:, :cols] = dev(x).to(dtype)
    want_q, want_s = of.quant_int8_rows(x)
    q, intact = _guarded(rows, cols, I8)
    got_q, got_s = fp8q.int8_quant_rows(buf[:, :cols], q=q)
    assert_bytes_equal(host(got_s), want_s, "scales")
    assert_bytes_equal(host(got_q), want_q, "codes")
    intact()
    q2, s2 = fp8q.int8_quant_rows(buf[:, :cols])          # outputs of the binding
    assert q2.shape == (rows, cols) and torch.equal(q2, got_q) and torch.equal(s2, got_s)


def test_int8_quant_rows_exact_steps():
    """Halves round to even, the whole range is reached, and the largest floats do not overflow."""
    fp8q = require_gpu()
    x = np.zeros((3, 300), np.float32)
    x[0] = np.arange(300) - 150
    x[0, 0] = 254.0                                       # scale 2: every odd value is a tie
    x[1, :4] = [3.0e38, -3.0e38, 1.5e38, 1.0]
    x[2, :3] = [2.0 ** -126, -2.0 ** -127, 2.0 ** -149]   # below the floor: codes of a scale 2^-126
    want_q, want_s = of.quant_int8_rows(x)
    q, s = fp8q.int8_quant_rows(dev(x))
    assert_bytes_equal(host(s), want_s, "scales")
    assert_bytes_equal(host(q)[:2], want_q[:2], "codes")
    assert host(q)[2, 0] == 1 and not host(q)[2, 3:].any()


def test_int8_quant_rows_empty():
    fp8q = require_gpu()
    q, s = fp8q.int8_quant_rows(torch.empty((0, 16), device="cuda"))
    assert q.shape == (0, 16) and s.shape == (0,)
    q, s = fp8q.int8_quant_rows(torch.empty((3, 0), device="cuda"))
    assert q.shape == (3, 0) and bool((s == 2.0 ** -126).all())


# ---------------------------------------------------------------------------
# int8_gemm, int8_gemm_gated
# ---------------------------------------------------------------------------
INT8_SIZES = [(1, 1, 1), (1, 16, 15), (1, 37, 16), (2, 3, 17), (15, 17, 63), (16, 16, 64), (17, 33, 65), (1, 130, 127),
              (33, 129, 128), (3, 48, 129), (64, 64, 1000), (65, 127, 1025), (128, 128, 640), (129, 255, 513),
              (200, 257, 2049), (256, 256, 1152), (257, 384, 333), (1, 300, 18432), (300, 1, 700), (513, 520, 272)]


def _int8_case(m, n, k, seed):
    rng = np.random.default_rng(seed)
    qa = rng.integers(-128, 128, size=(m, k)).astype(np.int8)
    qb = rng.integers(-128, 128, size=(n, k)).astype(np.int8)
    sa = np.exp2(rng.uniform(-9, -5, m)).astype(np.float32)
    sb = np.exp2(rng.uniform(-9, -5, n)).astype(np.float32)
    return qa, sa, qb, sb, normal_f32(rng, (n,), 1.0)


@pytest.mark.parametrize("m, n, k", INT8_SIZES)
@pytest.mark.parametrize("dtype, with_bias", [(BF, False), (F32, True)])
def test_int8_gemm(m, n, k, dtype, with_bias):
    fp8q = require_gpu()
    qa, sa, qb, sb, bias = _int8_case(m, n, k, m * 7 + n * 5 + k)
    a = _padded(qa, 113, ld=_up(k, 16) + 32)              # what lies between rows must not count
    b = _padded(qb, -119, offset=1)
    bias = bias if with_bias else None
    c, intact = _guarded(m, n, dtype)
    out = fp8q.int8_gemm(a, dev(sa), b, dev(sb), bias=None if bias is None else dev(bias), c=c)
    assert out.data_ptr() == c.data_ptr()
    ref = of.int8_gemm_ref(qa, sa, qb, sb, bias)
    prod = ref if bias is None else ref - bias.astype(np.float64)[None, :]
    _near(c, ref, 4 * U * (np.abs(prod) + np.abs(ref)) + TINY, dtype)
    intact()


@pytest.mark.parametrize("m, n, k", INT8_SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_int8_gemm_gated(m, n, k, act):
    fp8q = require_gpu()
    dtype = F32 if (m + n) % 2 else BF
    qa, sa, qb, sb, _ = _int8_case(m, 2 * n, k, m * 3 + n + k)
    sa = (sa * np.float32(8.0 / np.sqrt(k))).astype(np.float32)      # gates of a few units
    a, b = _padded(qa, 113), _padded(qb, -119)
    h, intact = _guarded(m, n, dtype)
    fp8q.int8_gemm_gated(a, dev(sa), b, dev(sb), act=act, h=h)
    gu = of.int8_gemm_ref(qa, sa, qb, sb)
    g, u = gu[:, :n], gu[:, n:]
    ref = of.gated(g, u, act)
    _near(h, ref, (22 + 20 * np.abs(_t(g, act))) * U * np.abs(ref) + TINY * (1 + np.abs(g * u)), dtype)
    intact()


@pytest.mark.parametrize("m", [1, 80, 300])
def test_int8_gemm_largest_sum(m):
    """All codes at -128 with the largest K: the sum, 128 * 128 * 131056, is 262144 short of 2^31."""
    fp8q = require_gpu()
    k, n = 131056, 48
    a = torch.full((m, k), -128, dtype=I8, device="cuda")
    b = torch.full((n, k), -128, dtype=I8, device="cuda")
    b[1] = 127
    one = torch.ones(max(m, n), device="cuda")
    c = _f64(fp8q.int8_gemm(a, one[:m], b, one[:n], out_dtype=F32))
    assert np.all(c[:, 0] == np.float32(128 * 128 * k)) and np.all(c[:, 1] == np.float32(-128 * 127 * k))


@pytest.mark.parametrize("gated", [False, True])
def test_int8_products_empty(gated):
    fp8q = require_gpu()
    fn = fp8q.int8_gemm_gated if gated else fp8q.int8_gemm
    for m, n, k in [(0, 32, 64), (5, 0, 64), (5, 32, 0)]:
        a, b = torch.empty((m, k), dtype=I8, device="cuda"), torch.empty((n, k), dtype=I8, device="cuda")
        c = fn(a, torch.ones(m, device="cuda"), b, torch.ones(n, device="cuda"), out_dtype=F32)
        assert c.shape == (m, n // 2 if gated else n) and not c.any()
    c = fp8q.int8_gemm(torch.empty((3, 0), dtype=I8, device="cuda"), torch.ones(3, device="cuda"),
                       torch.empty((5, 0), dtype=I8, device="cuda"), torch.ones(5, device="cuda"),
                       bias=torch.arange(5.0, device="cuda"), out_dtype=F32)
    assert torch.equal(c, torch.arange(5.0, device="cuda").expand(3, 5))


def test_int8_gemm_one_row_of_an_odd_width():
    """A single row's leading dimension is its own width: only its storage has to hold whole 16-byte chunks."""
    fp8q = require_gpu()
    qa, sa, qb, sb, _ = _int8_case(1, 40, 1001, 9)
    buf = torch.full((1008,), 99, dtype=I8, device="cuda")
    buf[:1001] = dev(qa[0])
    c = fp8q.int8_gemm(buf[:1001].unsqueeze(0), dev(sa), _padded(qb, 1), dev(sb), out_dtype=F32)
    ref = of.int8_gemm_ref(qa, sa, qb, sb)
    _near(c, ref, 8 * U * np.abs(ref) + TINY, F32)


# ---------------------------------------------------------------------------
# fp8_gemm_gated
# ---------------------------------------------------------------------------
FP8_SIZES = [(1, 128, 128), (1, 256, 1152), (2, 128, 640), (16, 384, 256), (17, 128, 1024), (33, 256, 384),
             (64, 128, 128), (100, 256, 512), (128, 128, 256), (129, 384, 640), (256, 256, 384), (300, 640, 256),
             (513, 384, 128), (777, 256, 512)]


def _fp8_case(m, f, k, seed):
    d = random_fp8_operands(seed, m, 2 * f, k, scale_lo=2.0 ** -10, scale_hi=2.0 ** -7)
    d["sa"] = (d["sa"] * np.float32(25.0 / np.sqrt(k))).astype(np.float32)       # gates of a few units
    return d


@pytest.mark.parametrize("m, f, k", FP8_SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_fp8_gemm_gated_f32(m, f, k, act):
    """FP32 gate and up against the exact product; h against act(g) * u of that same gate and up."""
    fp8q = require_gpu()
    d = _fp8_case(m, f, k, m + f + k)
    h, h_intact = _guarded(m, f, F32)
    gu, gu_intact = _guarded(m, 2 * f, F32)
    fp8q.fp8_gemm_gated(dev(d["qa"]), dev(d["sa"]), dev(d["qb"]), dev(d["sb"]), act=act, h=h, gu=gu)
    got = _f64(gu)
    assert og.rel_frobenius(got, og.gemm_ref(d["qa"], d["sa"], d["qb"], d["sb"], og.FPROP)) <= 2e-4
    g, u = got[:, :f], got[:, f:]
    assert np.abs(g).max() > 0.5
    ref = of.gated(g, u, act)
    _near(h, ref, (18 + 8 * np.abs(_t(g, act))) * U * np.abs(ref) + TINY * (1 + np.abs(g * u)), F32)
    h_intact()
    gu_intact()
    only = fp8q.fp8_gemm_gated(dev(d["qa"]), dev(d["sa"]), dev(d["qb"]), dev(d["sb"]), act=act, out_dtype=F32)
    assert torch.equal(only, h), "h depends on whether gate and up are kept"


@pytest.mark.parametrize("m, f, k", [(1, 128, 256), (50, 256, 384), (300, 384, 512), (512, 256, 1024)])
def test_fp8_gemm_gated_bf16(m, f, k):
    """BF16 outputs are the FP32 ones rounded once; operands are strided views."""
    fp8q = require_gpu()
    d = _fp8_case(m, f, k, m * 2 + f + k)
    a = torch.full((m, k + 48), 0x7F, dtype=torch.uint8, device="cuda")       # NaN codes between the rows
    b = torch.full((2 * f, k + 16), 0xFF, dtype=torch.uint8, device="cuda")
    a[:, :k], b[:, :k] = dev(d["qa"]), dev(d["qb"])
    args = (a[:, :k], dev(d["sa"]), b[:, :k].view(torch.float8_e4m3fn), dev(d["sb"]))
    h, gu = fp8q.fp8_gemm_gated(*args, save_gate_up=True)
    h32, gu32 = fp8q.fp8_gemm_gated(*args, out_dtype=F32, save_gate_up=True)
    assert torch.equal(h, h32.to(BF)) and torch.equal(gu, gu32.to(BF))
    ref = og.gemm_ref(d["qa"], d["sa"], d["qb"], d["sb"], og.FPROP)
    assert og.rel_frobenius(_f64(gu), og.round_bf16(ref)) <= 1e-3


# Rows and columns on both sides of the limits between kernels.  Which size chooses which kernel, and a size for every
# one of them: tests/ffn_kernel_sizes.py.
VARIANTS = [(2040, 17348), (2000, 5300), (1300, 5000), (500, 7000), (500, 3000), (200, 1000), (3, 5000), (9, 6200), (30, 6200),
            (40, 6200), (30, 3000), (20, 8000), (60, 8000), (40, 3000)]


@pytest.mark.parametrize("m, n", VARIANTS)
@pytest.mark.parametrize("k", [1101, 128])
@pytest.mark.parametrize("gated", [False, True])
def test_int8_every_variant(m, n, k, gated):
    """Against the same product in 64 bits on the GPU (integers there are exact)."""
    fp8q = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    rnd = lambda r, c: torch.randint(-128, 128, (r, _up(c, 16)), generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
    f = n // 2
    rows = 2 * f if gated else n
    a, b = rnd(m, k)[:, :k], rnd(rows, k)[:, :k]
    sa = torch.rand(m, generator=gen, device="cuda") * (4.0 / (5000 * k ** 0.5)) + 1e-7
    sb = torch.rand(rows, generator=gen, device="cuda") + 0.5
    y = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()[None, :]
    if gated:
        c, intact = _guarded(m, f, BF)
        fp8q.int8_gemm_gated(a, sa, b, sb, act=of.GELU_TANH, h=c)
        gu = _f64(y)
        g, u = gu[:, :f], gu[:, f:]
        ref = of.gated(g, u, of.GELU_TANH)
        _near(c, ref, (22 + 20 * np.abs(_t(g, of.GELU_TANH))) * U * np.abs(ref) + TINY * (1 + np.abs(g * u)), BF)
    else:
        bias = torch.randn(n, generator=gen, device="cuda")
        c, intact = _guarded(m, n, F32)
        fp8q.int8_gemm(a, sa, b, sb, bias=bias, c=c)
        ref = _f64(y + bias.double()[None, :])
        _near(c, ref, 4 * U * (np.abs(_f64(y)) + np.abs(ref)) + TINY, F32)
    intact()


@pytest.mark.parametrize("m, f", [(2040, 8704), (2000, 2688), (1300, 2560), (500, 3584), (500, 1536), (200, 512), (3, 2560), (30, 3200),
                                  (60, 4096), (20, 12160), (60, 2944)])
@pytest.mark.parametrize("k", [1152, 128])
def test_fp8_gated_every_variant(m, f, k):
    """Gate and up against the product of the dequantized codes in 64 bits on the GPU, and h against them."""
    fp8q = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(m + f + k)
    x = torch.randn((m, k), generator=gen, device="cuda")
    w = torch.randn((2 * f, k), generator=gen, device="cuda") * (1.5 / k ** 0.5)
    qa, sa = fp8q.fp8_quant_tile(x, fp8q.TILE_1x128, fp8q.MAXABS)
    qb, sb = fp8q.fp8_quant_block(w, fp8q.MAXABS)
    h, h_intact = _guarded(m, f, F32)
    gu, gu_intact = _guarded(m, 2 * f, F32)
    fp8q.fp8_gemm_gated(qa, sa, qb, sb, h=h, gu=gu)
    a = qa.view(torch.float8_e4m3fn).double() * sa.double().t().repeat_interleave(128, 1)
    b = qb.view(torch.float8_e4m3fn).double() * sb.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    ref = a @ b.t()
    rows = ((gu.double() - ref).norm(dim=1) / ref.norm(dim=1)).max().item()
    cols = ((gu.double() - ref).norm(dim=0) / ref.norm(dim=0)).max().item()
    assert rows <= 2e-4 and (m < 100 or cols <= 2e-4), (rows, cols)
    g, u = _f64(gu)[:, :f], _f64(gu)[:, f:]
    want = of.gated(g, u, of.SILU)
    _near(h, want, (18 + 8 * np.abs(g)) * U * np.abs(want) + TINY * (1 + np.abs(g * u)), F32)
    h_intact()
    gu_intact()


# (Of these, 500 rows run in 128x128 tiles by two teams and 200 in 64x64 by two; four teams: tests/ffn_kernel_sizes.py.)
@pytest.mark.parametrize("m, n", [(500, 7000), (200, 1000)])
@pytest.mark.parametrize("gated", [False, True])
def test_int8_teams_on_longer_k(m, n, gated):
    """Two teams of waves in 128x128 tiles, four in 64x64: chosen from about 2000 on."""
    test_int8_every_variant(m, n, 2300, gated)


@pytest.mark.parametrize("m, f", [(500, 3584), (200, 512)])
def test_fp8_gated_teams_on_longer_k(m, f):
    test_fp8_gated_every_variant(m, f, 2304)


@pytest.mark.parametrize("m, n", [(4200, 4059), (3300, 5700)])
@pytest.mark.parametrize("gated", [False, True])
def test_int8_round_and_a_few_tiles(m, n, gated):
    """A few 256x256 tiles more than one for each CU, the last ones not a whole number of columns."""
    test_int8_every_variant(m, n, 1101, gated)


@pytest.mark.parametrize("m, f", [(1, 2048), (16, 2043), (17, 2041), (32, 2048), (32, 2049)])
def test_int8_gated_eight_columns_a_workgroup(m, f):
    """Up to 2048 columns, odd ones too: a workgroup has 8, gate and up in one fragment; 2049 are one too many."""
    test_int8_every_variant(m, 2 * f, 1101, True)


@pytest.mark.parametrize("m, f", [(1, 2048), (16, 1920), (17, 2048), (32, 1408)])
def test_fp8_gated_eight_columns_a_workgroup(m, f):
    test_fp8_gated_every_variant(m, f, 1152)


def test_fp8_gated_round_and_a_few_tiles():
    test_fp8_gated_every_variant(4200, 2048, 1152)


def test_fp8_gemm_gated_saturated_gates():
    """Gates of thousands on both sides: sigma is exactly 0 or 1 there and nothing overflows to NaN."""
    fp8q = require_gpu()
    d = _fp8_case(40, 128, 256, 5)
    sa = dev(d["sa"]) * 1e4
    for act in ACTS:
        h, gu = fp8q.fp8_gemm_gated(dev(d["qa"]), sa, dev(d["qb"]), dev(d["sb"]), act=act, out_dtype=F32,
                                    save_gate_up=True)
        g, u = _f64(gu)[:, :128], _f64(gu)[:, 128:]
        ref = of.gated(g, u, act)
        assert bool(torch.isfinite(h).all()) and np.abs(g).max() > 1e4
        _near(h, ref, (18 + 8 * np.minimum(np.abs(_t(g, act)), 200)) * U * np.abs(ref) + TINY * (1 + np.abs(g * u)), F32)


def test_fp8_gemm_gated_empty():
    fp8q = require_gpu()
    e = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")      # noqa: E731
    z = lambda *s: torch.ones(s, device="cuda")                          # noqa: E731
    assert fp8q.fp8_gemm_gated(e(0, 128), z(1, 0), e(256, 128), z(2, 1)).shape == (0, 128)
    h, gu = fp8q.fp8_gemm_gated(e(3, 0), z(0, 3), e(256, 0), z(2, 0), save_gate_up=True)
    assert h.shape == (3, 128) and not h.any() and not gu.any()


# ---------------------------------------------------------------------------
# fp8_gated_backward
# ---------------------------------------------------------------------------
BWD_SIZES = [(1, 128), (3, 256), (127, 128), (128, 384), (129, 256), (300, 128), (513, 640)]


def _bwd_case(m, f, seed, sigma=2.0):
    rng = np.random.default_rng(seed)
    rnd = lambda x: bf16_bits_as_f32(to_bf16_bits(x))                    # noqa: E731
    dh = rnd(normal_f32(rng, (m, f), 1e-3))
    gu = rnd(add_outliers(rng, normal_f32(rng, (m, 2 * f), sigma), 0.002, 20.0))
    return dh, gu


@pytest.mark.parametrize("m, f", BWD_SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_gradient(m, f, act):
    """D itself against the formula and against differences of the 64-bit forward pass."""
    fp8q = require_gpu()
    dh, gu = _bwd_case(m, f, m + f + act)
    d, intact = _guarded(m, 2 * f, F32)
    fp8q.fp8_gated_backward(dev(dh), dev(gu), act=act, dgu=d)
    intact()
    g, u = gu[:, :f].astype(np.float64), gu[:, f:].astype(np.float64)
    t = np.abs(_t(g, act))
    dg, du = of.gated_backward(dh, g, u, act)
    a = np.abs(of.act(g, act) * dh)
    _near(_f64(d)[:, f:], du, (18 + 8 * np.minimum(t, 200)) * U * a + TINY, F32)
    s = np.abs(of._logistic(_t(g, act)))
    terms = s + np.abs(of.act_slope(g, act) - of._logistic(_t(g, act)))
    tol = (20 + 8 * np.minimum(t, 200)) * U * terms * np.abs(dh * u)
    _near(_f64(d)[:, :f], dg, tol + TINY, F32)
    # central differences with step 1e-5: truncation under 4e-11 and rounding under |act| 2^-51 / 1e-5 per unit of dh u
    e = 1e-5
    num = dh * u * (of.act(g + e, act) - of.act(g - e, act)) / ((g + e) - (g - e))
    _near(_f64(d)[:, :f], num, tol + TINY + np.abs(dh * u) * (1e-10 + 1e-10 * np.abs(g)), F32)


@pytest.mark.parametrize("m, f", BWD_SIZES)
@pytest.mark.parametrize("mode", [0, 1])
def test_gated_backward_codes(m, f, mode):
    """The codes and scales are those of the FP32 gradient, quantized in both tilings over whole 128-row tiles, and
    BF16 inputs give what the same values in FP32 give, bit for bit."""
    fp8q = require_gpu()
    act, mp = (m + mode) % 2, _up(m, 128)
    dh, gu = _bwd_case(m, f, 11 * m + f)
    d = torch.empty((m, 2 * f), device="cuda")
    out = fp8q.fp8_gated_backward(dev(dh), dev(gu), act=act, mode=mode, dgu=d)
    full = np.zeros((mp, 2 * f), np.float32)
    full[:m] = host(d)
    name = "pow2" if mode else "maxabs"
    want = oq.quant_1x128(full, name) + oq.quant_128x1(full, name)
    for got, ref, what in zip(out, want, ("1x128 codes", "1x128 scales", "128x1 codes", "128x1 scales")):
        assert_bytes_equal(host(got), ref, what)
    d16 = torch.empty((m, 2 * f), dtype=BF, device="cuda")
    out16 = fp8q.fp8_gated_backward(dev(dh).to(BF), dev(gu).to(BF), act=act, mode=mode, dgu=d16)
    assert all(torch.equal(x, y) for x, y in zip(out, out16)) and torch.equal(d16, d.to(BF))


def test_gated_backward_strided_and_guarded():
    fp8q = require_gpu()
    m, f = 200, 256
    dh, gu = _bwd_case(m, f, 77)
    want = fp8q.fp8_gated_backward(dev(dh), dev(gu))
    bh = torch.full((m, f + 8), float("nan"), device="cuda")
    bg = torch.full((m, 2 * f + 12), float("nan"), device="cuda")
    bh[:, :f], bg[:, :2 * f] = dev(dh), dev(gu)
    q = torch.full((258, 2 * f + 16), 0x55, dtype=torch.uint8, device="cuda")
    qt = torch.full((2 * f + 2, 272), 0x55, dtype=torch.uint8, device="cuda")
    got = fp8q.fp8_gated_backward(bh[:, :f], bg[:, :2 * f], q=q[1:257, :2 * f], q_t=qt[1:2 * f + 1, :256])
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    q[1:257, :2 * f] = 0x55
    qt[1:2 * f + 1, :256] = 0x55
    assert bool((q == 0x55).all()) and bool((qt == 0x55).all()), "written outside the output"


@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_extreme_gates(act):
    """Gates from 1e-30 to 3e38 on both sides: finite gradients, exactly 0 or the identity's where sigma saturates."""
    fp8q = require_gpu()
    g = np.array([0.0, -0.0, 1e-30, -1e-30, 90, -90, 200, -200, 1e5, -1e5, 1e20, -1e20, 3e38, -3e38], np.float32)
    gu = np.ones((len(g), 256), np.float32)
    gu[:, :128] = g[:, None]
    d = torch.empty((len(g), 256), device="cuda")
    fp8q.fp8_gated_backward(torch.full((len(g), 128), 0.5, device="cuda"), dev(gu), act=act, dgu=d)
    dg, du = of.gated_backward(0.5, np.minimum(np.maximum(g.astype(np.float64), -1e6), 1e6), 1.0, act)
    _near(_f64(d)[:, 0], dg, (20 + 8 * np.minimum(np.abs(_t(g, act)), 200)) * U * np.maximum(np.abs(dg), 1) + TINY, F32)
    act_ref = np.where(g > 100, g, np.where(g < -100, 0.0, of.act(np.clip(g, -100, 100).astype(np.float64), act)))
    _near(_f64(d)[:, 128], 0.5 * act_ref, (18 + 8 * np.minimum(np.abs(_t(g, act)), 200)) * U * np.abs(act_ref) + TINY, F32)


def test_gated_backward_empty():
    fp8q = require_gpu()
    q, s, qt, st = fp8q.fp8_gated_backward(torch.empty((0, 128), device="cuda"), torch.empty((0, 256), device="cuda"))
    assert q.shape == (0, 256) and s.shape == (2, 0) and qt.shape == (256, 0) and st.shape == (0, 256)


# ---------------------------------------------------------------------------
# Refusals of the binding, streams, replay
# ---------------------------------------------------------------------------
def test_binding_refusals():
    fp8q = require_gpu()
    i8 = lambda *s: torch.zeros(s, dtype=I8, device="cuda")              # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")     # noqa: E731
    f = lambda *s: torch.zeros(s, device="cuda")                         # noqa: E731
    with pytest.raises(TypeError, match="a must be torch.int8"):
        fp8q.int8_gemm(u8(4, 32), f(4), i8(8, 32), f(8))
    with pytest.raises(ValueError, match="disagree on K"):
        fp8q.int8_gemm(i8(4, 32), f(4), i8(8, 48), f(8))
    with pytest.raises(ValueError, match="b_scales has shape"):
        fp8q.int8_gemm(i8(4, 32), f(4), i8(8, 32), f(7))
    with pytest.raises(ValueError, match="bias has shape"):
        fp8q.int8_gemm(i8(4, 32), f(4), i8(8, 32), f(8), bias=f(1, 8))
    with pytest.raises(TypeError, match="c must be bfloat16 or float32"):
        fp8q.int8_gemm(i8(4, 32), f(4), i8(8, 32), f(8), out_dtype=torch.float16)
    with pytest.raises(ValueError, match="16-byte chunks"):
        fp8q.int8_gemm(i8(1, 33), f(1), i8(8, 48)[:, :33], f(8))       # the storage ends inside a chunk
    with pytest.raises(fp8q.Fp8qError) as e:
        fp8q.int8_gemm(i8(4, 40), f(4), i8(8, 40), f(8))               # rows 40 bytes apart
    assert e.value.status == fp8q.ERR_ALIGN
    with pytest.raises(ValueError, match="as many gate rows as up rows"):
        fp8q.int8_gemm_gated(i8(4, 32), f(4), i8(7, 32), f(7))
    with pytest.raises(ValueError, match="h has shape"):
        fp8q.int8_gemm_gated(i8(4, 32), f(4), i8(8, 32), f(8), h=f(4, 8))
    with pytest.raises(ValueError, match="must be a device tensor"):
        fp8q.int8_gemm_gated(i8(4, 32), f(4), i8(8, 32).cpu(), f(8))
    with pytest.raises(ValueError, match="scales has shape"):
        fp8q.int8_quant_rows(f(4, 32), scales=f(32))
    with pytest.raises(ValueError, match="row-major"):
        fp8q.int8_quant_rows(f(32, 4).t())
    with pytest.raises(TypeError, match="unsupported dtype"):
        fp8q.int8_quant_rows(f(4, 32).half())
    with pytest.raises(ValueError, match="a_scales has shape"):
        fp8q.fp8_gemm_gated(u8(4, 128), f(4, 1), u8(256, 128), f(2, 1))
    with pytest.raises(TypeError, match="gu must be"):
        fp8q.fp8_gemm_gated(u8(4, 128), f(1, 4), u8(256, 128), f(2, 1), gu=f(4, 256))
    with pytest.raises(fp8q.Fp8qError) as e:
        fp8q.fp8_gemm_gated(u8(4, 128), f(1, 4), u8(192, 128), f(2, 1))
    assert e.value.status == fp8q.ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="gu has shape"):
        fp8q.fp8_gated_backward(f(4, 128), f(4, 128))
    with pytest.raises(TypeError, match="gu must be"):
        fp8q.fp8_gated_backward(f(4, 128), f(4, 256).to(BF))
    with pytest.raises(ValueError, match="q_t has shape"):
        fp8q.fp8_gated_backward(f(4, 128), f(4, 256), q_t=u8(256, 4))
    with pytest.raises(ValueError, match="scales has shape"):
        fp8q.fp8_gated_backward(f(4, 128), f(4, 256), scales=f(2, 4))


def _chain(fp8q, x, w, wd, dh, stream=None):
    """Every operator once, from BF16 inputs."""
    qx, sx = fp8q.fp8_quant_tile(x, fp8q.TILE_1x128, fp8q.MAXABS, stream=stream)
    qw, sw = fp8q.fp8_quant_block(w, fp8q.MAXABS, stream=stream)
    h, gu = fp8q.fp8_gemm_gated(qx, sx, qw, sw, save_gate_up=True, stream=stream)
    back = fp8q.fp8_gated_backward(dh, gu, stream=stream)
    ix, isx = fp8q.int8_quant_rows(x, stream=stream)
    iw, isw = fp8q.int8_quant_rows(w, stream=stream)
    ih = fp8q.int8_gemm_gated(ix, isx, iw, isw, stream=stream)
    qh, sh = fp8q.int8_quant_rows(ih, stream=stream)
    qd, sd = fp8q.int8_quant_rows(wd, stream=stream)
    return (h, gu, *back, ih, fp8q.int8_gemm(qh, sh, qd, sd, stream=stream))


def _chain_inputs(seed, m, k=384, f=256):
    rng = np.random.default_rng(seed)
    r = lambda *s, sigma=1.0: dev_bf16(to_bf16_bits(normal_f32(rng, s, sigma)))   # noqa: E731
    return r(m, k), r(2 * f, k, sigma=0.05), r(k, f, sigma=0.05), r(m, f, sigma=1e-3)


@pytest.mark.parametrize("m", [3, 200])
def test_chain_on_a_user_stream(m):
    fp8q = require_gpu()
    args = _chain_inputs(31, m)
    want = [host(t.view(torch.uint8)) for t in _chain(fp8q, *args)]
    busy = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):                                    # the default stream is busy meanwhile
        busy = busy @ busy.t() * 1e-3
    with torch.cuda.stream(s):
        got = _chain(fp8q, *args, stream=s)
    s.synchronize()
    for x, y in zip(got, want):
        assert np.array_equal(host(x.view(torch.uint8)), y)


@pytest.mark.parametrize("m", [1, 200])
def test_chain_captured_in_a_hip_graph_and_replayed(m):
    fp8q = require_gpu()
    bufs = _chain_inputs(41, m)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _chain(fp8q, *bufs)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _chain(fp8q, *bufs)
    torch.cuda.synchronize()
    for seed in (51, 52, 53):
        args = _chain_inputs(seed, m)
        want = [host(t.view(torch.uint8)) for t in _chain(fp8q, *args)]
        for b, x in zip(bufs, args):
            b.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert np.array_equal(host(x.view(torch.uint8)), y), seed
