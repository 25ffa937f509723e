"""Gated feed-forward operators on tensors beyond 2^31 elements or bytes and at the largest leading dimension: every
address past the 32-bit range is formed correctly.  Inputs are drawn on the GPU (seeded); the 64-bit definitions
recompute sampled rows and columns on both sides of the limit."""

import numpy as np
import pytest
import torch

from oracle import ffn as of, gemm as og, quant as oq
from tests.helpers import assert_bytes_equal, host, require_gpu
from workloads import device_fp8_codes

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF, I8 = torch.float32, torch.bfloat16, torch.int8
LD_MAX = (1 << 31) // 512 - 128          # the largest operand leading dimension the C ABI accepts (bytes)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _int8(seed, rows, cols):
    return torch.randint(-128, 128, (rows, cols), generator=_gen(seed), device="cuda", dtype=I8)


def _scales(seed, shape, lo, hi):
    return torch.exp2(torch.rand(shape, generator=_gen(seed), device="cuda") * (hi - lo) + lo)


def _f64(t):
    return t.double().cpu().numpy()


def test_outputs_beyond_2g_elements():
    """40000 x 2 x 32768 pre-activations (2.6e9), then their gradient in both tilings: sampled rows and columns."""
    fp8q = require_gpu()
    m, f, k = 40000, 32768, 128
    qa, qb = device_fp8_codes(1, (m, k)), device_fp8_codes(2, (2 * f, k))
    sa, sb = _scales(3, (1, m), -12, -10), _scales(4, (2 * f // 128, 1), -4, -3)
    h, gu = fp8q.fp8_gemm_gated(qa, sa, qb, sb, save_gate_up=True)
    rows = np.array([0, 32767, 32768, 32769, m - 1])                         # row 32768 of gu starts at element 2^31
    ref = og.gemm_ref(host(qa[rows]), host(sa[:, rows]), host(qb), host(sb), og.FPROP)
    got = _f64(gu[rows])
    assert og.rel_frobenius(got, og.round_bf16(ref)) <= 1e-3
    # h comes from the unrounded gate and up: within what rounding them and h to BF16 explains, 2^-9 each and the
    # gate's amplified by 1 + |g|
    g, u = got[:, :f], got[:, f:]
    want = of.gated(g, u, of.SILU)
    assert np.all(np.abs(_f64(h[rows]) - want) <= (3 + np.abs(g)) * 2.0 ** -8 * np.abs(want) + 1e-30)

    q, s, q_t, s_t = fp8q.fp8_gated_backward(h, gu)
    band = 32768 // 128                                                      # rows 32768..32895: past element 2^31
    one = fp8q.fp8_gated_backward(h[32768:32896].contiguous(), gu[32768:32896].contiguous())
    assert torch.equal(q[32768:32896], one[0]) and torch.equal(s[:, 32768:32896], one[1])
    assert torch.equal(q_t[:, 32768:32896], one[2]) and torch.equal(s_t[band:band + 1], one[3])
    gg, uu, dh = _f64(gu[32768:32896, :f]), _f64(gu[32768:32896, f:]), _f64(h[32768:32896])
    dg, du = of.gated_backward(dh, gg, uu, of.SILU)
    d = np.concatenate([dg, du], axis=1).astype(np.float32)
    codes, scales = oq.quant_1x128(d, "maxabs")
    # FP32 rounding of D moves a code where it lies next to a step's edge: nearly all agree
    assert np.mean(host(one[0]) == codes) >= 0.9999
    assert np.max(np.abs(host(one[1]) / scales - 1)) <= 64 * U
    del h, gu, q, s, q_t, s_t
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m", [1, 20, 300])
def test_int8_weight_beyond_2g_bytes(m):
    """B of 139264 x 16384 (2.28e9 bytes), streamed and tiled: columns on both sides of byte 2^31."""
    fp8q = require_gpu()
    n, k = 139264, 16384
    a, b = _int8(11, m, k), _int8(12, n, k)
    sa, sb = _scales(13, (m,), -12, -8), _scales(14, (n,), -12, -8)
    cols = np.array([0, 131071, 131072, 131073, n - 1])                      # row 131072 of B starts at byte 2^31
    c = fp8q.int8_gemm(a, sa, b, sb, out_dtype=F32)
    ref = of.int8_gemm_ref(host(a), host(sa), host(b[cols]), host(sb[cols]))
    assert np.all(np.abs(_f64(c[:, cols]) - ref) <= 8 * U * np.abs(ref) + 1e-30)
    h = fp8q.int8_gemm_gated(a, sa * 2.0 ** -4, b, sb, out_dtype=F32)
    f = n // 2
    pick = np.array([0, 61439, 61440, 61441, f - 1])                         # up row f + 61440 = 131072
    gu = of.int8_gemm_ref(host(a), host(sa * 2.0 ** -4), host(b[np.r_[pick, f + pick]]), host(sb[np.r_[pick, f + pick]]))
    g, u = gu[:, :5], gu[:, 5:]
    want = of.gated(g, u, of.SILU)
    assert np.all(np.abs(_f64(h[:, pick]) - want) <= (22 + 20 * np.abs(g)) * U * np.abs(want) + 1e-30)
    del a, b, c, h
    torch.cuda.empty_cache()


def test_int8_rows_beyond_2g_elements():
    """139264 x 16384 (2.28e9 elements): rows on both sides of 2^31, and those codes as the A operand."""
    fp8q = require_gpu()
    m, k, n = 139264, 16384, 96
    x = torch.randn((m, k), generator=_gen(21), device="cuda", dtype=BF)
    q, s = fp8q.int8_quant_rows(x)
    rows = np.array([0, 131071, 131072, m - 1])
    want_q, want_s = of.quant_int8_rows(x[rows].float().cpu().numpy())
    assert_bytes_equal(host(q[rows]), want_q, "codes")
    assert_bytes_equal(host(s[rows]), want_s, "scales")
    b, sb = _int8(22, n, k), _scales(23, (n,), -12, -8)
    c = fp8q.int8_gemm(q, s, b, sb, out_dtype=F32)
    ref = of.int8_gemm_ref(want_q, want_s, host(b), host(sb))
    assert np.all(np.abs(_f64(c[rows]) - ref) <= 8 * U * np.abs(ref) + 1e-30)
    del x, q, b, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m", [9, 300])
def test_largest_leading_dimension(m):
    """Rows 4,194,176 bytes apart, the most the C ABI accepts; the bytes between them must not count."""
    fp8q = require_gpu()
    k, f = 384, 128

    def spread(t, fill):
        buf = torch.full((t.shape[0], LD_MAX), fill, dtype=t.dtype, device="cuda")
        buf[:, :t.shape[1]] = t
        return buf[:, :t.shape[1]]
    a, b = _int8(31, m, k - 3), _int8(32, 2 * f, k - 3)
    sa, sb = _scales(33, (m,), -9, -8), _scales(34, (2 * f,), -9, -8)
    c = fp8q.int8_gemm(spread(a, 77), sa, spread(b, -77), sb, out_dtype=F32)
    ref = of.int8_gemm_ref(host(a), host(sa), host(b), host(sb))
    assert np.all(np.abs(_f64(c) - ref) <= 8 * U * np.abs(ref) + 1e-30)
    qa, qb = device_fp8_codes(35, (m, k)), device_fp8_codes(36, (2 * f, k))
    ta, tb = _scales(37, (k // 128, m), -10, -8), _scales(38, (2 * f // 128, k // 128), -8, -6)
    args = (spread(qa, 0x7F), ta, spread(qb, 0xFF), tb)
    h, gu = fp8q.fp8_gemm_gated(*args, out_dtype=F32, save_gate_up=True)
    ref = og.gemm_ref(host(qa), host(ta), host(qb), host(tb), og.FPROP)
    assert og.rel_frobenius(_f64(gu), ref) <= 2e-4 and bool(torch.isfinite(h).all())
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m, f, k", [(3, 640, 1000), (200, 500, 3000), (500, 1500, 1111), (900, 2650, 640)])
def test_two_calls_give_the_same_bytes(m, f, k):
    """Sums of waves and teams are joined in a fixed order."""
    fp8q = require_gpu()
    a, b = _int8(41, m, -(-k // 16) * 16)[:, :k], _int8(42, 2 * f, -(-k // 16) * 16)[:, :k]
    sa, sb = _scales(43, (m,), -12, -11), _scales(44, (2 * f,), -9, -8)
    x, y = (fp8q.int8_gemm_gated(a, sa, b, sb, out_dtype=F32) for _ in range(2))
    assert torch.equal(x, y)
    k8, f8 = -(-k // 128) * 128, -(-f // 128) * 128
    qa, qb = device_fp8_codes(45, (m, k8)), device_fp8_codes(46, (2 * f8, k8))
    ta, tb = _scales(47, (k8 // 128, m), -14, -12), _scales(48, (2 * f8 // 128, k8 // 128), -8, -6)
    first, second = (fp8q.fp8_gemm_gated(qa, ta, qb, tb, out_dtype=F32, save_gate_up=True) for _ in range(2))
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
