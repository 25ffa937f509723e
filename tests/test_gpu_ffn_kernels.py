"""Every kernel of the gated and the 8-bit integer products at sizes that choose it (tests/ffn_kernel_sizes.py), in
both output types, against 64 bits on the GPU.  Tolerances are those derived in tests/test_gpu_ffn.py; a BF16 result is
the FP32 one of the same kernel rounded once, so it has to equal that exactly."""

import math

import pytest
import torch

from tests.ffn_kernel_sizes import FP8_GATED, INT8, INT8_GATED
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

U, TINY = 2.0 ** -24, 2.0 ** -100
F32, BF = torch.float32, torch.bfloat16


def _out(rows, cols, dtype):
    """An output view among sentinels, whose rows fill whole 128-byte lines in BF16 (they are stored another way than
    partial ones), and a check that nothing around it changed."""
    per = 64 if dtype == BF else 4
    ld = -(-cols // per) * per + per
    buf = torch.full((rows + 2, ld), -77, dtype=dtype, device="cuda")

    def intact():
        b = buf.clone()
        b[1:rows + 1, :cols] = -77
        assert bool((b == -77).all()), "written outside the output"
    return buf[1:rows + 1, :cols], intact


def _near(got, ref, tol):
    bad = ~((got.double() - ref).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(x[0]) for x in torch.nonzero(bad, as_tuple=True))
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i].item()!r} want "
                             f"{ref[i].item()!r} +- {tol[i].item()!r}")


def _gelu(g):
    """GELU's tanh form as a logistic, and the logistic's argument."""
    t = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(t), t


def _int8(m, rows, k):
    gen = torch.Generator(device="cuda").manual_seed(m + rows + k)
    ld = -(-k // 16) * 16
    rnd = lambda r: torch.randint(-128, 128, (r, ld), generator=gen, device="cuda", dtype=torch.int8)[:, :k]  # noqa: E731
    sa = torch.rand(m, generator=gen, device="cuda") * (4.0 / (5000 * k ** 0.5)) + 1e-7
    return rnd(m), sa, rnd(rows), torch.rand(rows, generator=gen, device="cuda") + 0.5, gen


def _product(a, sa, b, sb):
    """The integer sum is exact in 64-bit floats."""
    return (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()[None, :]


@pytest.mark.parametrize("m, n, k, kernel", INT8)
def test_int8_gemm(m, n, k, kernel):
    fp8q = require_gpu()
    a, sa, b, sb, gen = _int8(m, n, k)
    bias = torch.randn(n, generator=gen, device="cuda")
    (c, c_ok), (h, h_ok) = _out(m, n, F32), _out(m, n, BF)
    fp8q.int8_gemm(a, sa, b, sb, bias=bias, c=c)
    fp8q.int8_gemm(a, sa, b, sb, bias=bias, c=h)
    prod = _product(a, sa, b, sb)
    ref = prod + bias.double()[None, :]
    _near(c, ref, 4 * U * (prod.abs() + ref.abs()) + TINY)
    assert torch.equal(h, c.to(BF))
    c_ok()
    h_ok()


@pytest.mark.parametrize("m, n, k, kernel", INT8_GATED)
def test_int8_gemm_gated(m, n, k, kernel):
    fp8q = require_gpu()
    a, sa, b, sb, _ = _int8(m, 2 * n, k)
    (c, c_ok), (h, h_ok) = _out(m, n, F32), _out(m, n, BF)
    for out in (c, h):
        fp8q.int8_gemm_gated(a, sa, b, sb, act=fp8q.ACT_GELU_TANH, h=out)
    gu = _product(a, sa, b, sb)
    g, u = gu[:, :n], gu[:, n:]
    act, t = _gelu(g)
    _near(c, act * u, (22 + 20 * t.abs()) * U * (act * u).abs() + TINY * (1 + (g * u).abs()))
    assert torch.equal(h, c.to(BF))
    c_ok()
    h_ok()


@pytest.mark.parametrize("m, f, k, kernel", FP8_GATED)
def test_fp8_gemm_gated(m, f, k, kernel):
    fp8q = require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(m + f + k)
    qa, sa = fp8q.fp8_quant_tile(torch.randn((m, k), generator=gen, device="cuda"), fp8q.TILE_1x128, fp8q.MAXABS)
    qb, sb = fp8q.fp8_quant_block(torch.randn((2 * f, k), generator=gen, device="cuda") * (1.5 / k ** 0.5), fp8q.MAXABS)
    (h, h_ok), (gu, gu_ok) = _out(m, f, F32), _out(m, 2 * f, F32)
    (h16, h16_ok), (gu16, gu16_ok) = _out(m, f, BF), _out(m, 2 * f, BF)
    fp8q.fp8_gemm_gated(qa, sa, qb, sb, act=fp8q.ACT_GELU_TANH, h=h, gu=gu)
    fp8q.fp8_gemm_gated(qa, sa, qb, sb, act=fp8q.ACT_GELU_TANH, h=h16, gu=gu16)
    a = qa.view(torch.float8_e4m3fn).double() * sa.double().t().repeat_interleave(128, 1)
    b = qb.view(torch.float8_e4m3fn).double() * sb.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    ref = a @ b.t()
    rows = ((gu.double() - ref).norm(dim=1) / ref.norm(dim=1)).max().item()
    cols = ((gu.double() - ref).norm(dim=0) / ref.norm(dim=0)).max().item()
    assert rows <= 2e-4 and (m < 100 or cols <= 2e-4), (rows, cols)
    g, u = gu[:, :f].double(), gu[:, f:].double()
    act, t = _gelu(g)
    _near(h, act * u, (18 + 8 * t.abs()) * U * (act * u).abs() + TINY * (1 + (g * u).abs()))
    assert torch.equal(h16, h.to(BF)) and torch.equal(gu16, gu.to(BF))
    for ok in (h_ok, gu_ok, h16_ok, gu16_ok):
        ok()
