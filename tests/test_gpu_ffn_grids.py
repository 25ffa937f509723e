"""Gated feed-forward operators on sizes that take more threads than one launch has (2^32)."""

import pytest
import torch

from oracle import ffn as of
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("rows, cols", [((1 << 28) + 5, 8), ((1 << 24) + 3, 1025)])
def test_int8_quant_rows_beyond_one_grid(rows, cols):
    """16 lanes a row and 2^28 rows, a workgroup a row and 2^24: the rows past one grid are a second round of it."""
    fp8q = require_gpu()
    ld, part = -(-cols // 8) * 8, 1 << 20 if cols == 8 else 1 << 16
    gen = torch.Generator(device="cuda").manual_seed(cols)
    base = torch.randn((part, ld), generator=gen, device="cuda", dtype=BF)
    x = torch.empty((rows, ld), device="cuda", dtype=BF)
    for r in range(0, rows, part):                       # the same rows again and again, in another order at the end
        n = min(part, rows - r)
        x[r:r + n] = base[:n] if n == part else base[part - n:]
    q, s = fp8q.int8_quant_rows(x[:, :cols])
    want_q, want_s = (torch.from_numpy(t).cuda() for t in of.quant_int8_rows(base[:, :cols].float().cpu().numpy()))
    for r in range(0, rows, part):
        n = min(part, rows - r)
        same = slice(0, n) if n == part else slice(part - n, part)
        assert torch.equal(q[r:r + n], want_q[same]) and torch.equal(s[r:r + n], want_s[same]), r
    del x, q, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m, n, gated", [(1, (1 << 27) + 40, False), (3, (1 << 27) + 24, True), (9, (1 << 28) + 200, False)])
def test_int8_products_of_more_columns_than_one_launch_takes(m, n, gated):
    """The streaming kernel's launches are cut along N (16 codes deep; 2^27 columns in workgroups of 16, 2^28 of 32)."""
    fp8q = require_gpu()
    k, part, rows = 16, 1 << 24, 2 * n if gated else n
    gen = torch.Generator(device="cuda").manual_seed(n % 1000)
    a = torch.randint(-128, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (rows, k), generator=gen, device="cuda", dtype=torch.int8)
    sa = torch.rand(m, generator=gen, device="cuda") * 1e-4 + 1e-5
    sb = torch.rand(rows, generator=gen, device="cuda") + 0.5
    if gated:
        got = fp8q.int8_gemm_gated(a, sa, b, sb, out_dtype=torch.float32)
    else:
        bias = torch.randn(n, generator=gen, device="cuda")
        got = fp8q.int8_gemm(a, sa, b, sb, bias=bias, out_dtype=torch.float32)
    for c in range(0, n, part):
        e = min(n, c + part)
        y = lambda lo: (a.double() @ b[lo + c:lo + e].double().t()) * sa.double()[:, None] * sb[lo + c:lo + e].double()  # noqa: E731
        # the tolerances of tests/test_gpu_ffn.py: the scaled sum to 4 units, the gated product to 22 + 20 |g|
        if gated:
            g, u = y(0), y(n)
            ref = g * torch.sigmoid(g) * u
            tol = (22 + 20 * g.abs()) * 2.0 ** -24 * ref.abs() + 2.0 ** -100 * (1 + (g * u).abs())
        else:
            prod = y(0)
            ref = prod + bias[c:e].double()
            tol = 4 * 2.0 ** -24 * (prod.abs() + ref.abs()) + 2.0 ** -100
        assert bool(((got[:, c:e].double() - ref).abs() <= tol).all()), c
    del b, got
    torch.cuda.empty_cache()


def test_int8_product_of_more_rows_than_one_launch_takes():
    """2^31 + 3 rows of one column: the tiled kernel's launches are cut along M."""
    fp8q = require_gpu()
    m, n, k, part = (1 << 31) + 3, 1, 16, 1 << 26
    gen = torch.Generator(device="cuda").manual_seed(5)
    base = torch.randint(-128, 128, (part + 7, k), generator=gen, device="cuda", dtype=torch.int8)
    scale = torch.rand(part + 7, generator=gen, device="cuda") + 0.5
    a, sa = torch.empty((m, k), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    b = torch.randint(-128, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    sb = torch.rand(n, generator=gen, device="cuda") + 0.5
    for i, r in enumerate(range(0, m, part)):              # the same rows, shifted by one of eight offsets each time
        e = min(m, r + part)
        a[r:e], sa[r:e] = base[i % 8:i % 8 + e - r], scale[i % 8:i % 8 + e - r]
    got = fp8q.int8_gemm(a, sa, b, sb, out_dtype=torch.bfloat16)
    ref = (base.double() @ b.double().t()) * scale.double()[:, None] * sb.double()
    tol = ref.abs() * (2.0 ** -8 + 8 * 2.0 ** -24) + 2.0 ** -100
    for i, r in enumerate(range(0, m, part)):
        e, o = min(m, r + part), i % 8
        assert bool(((got[r:e].double() - ref[o:o + e - r]).abs() <= tol[o:o + e - r]).all()), r
    del a, sa, got, ref, tol
    torch.cuda.empty_cache()


def test_fp8_gemm_gated_of_more_columns_than_one_launch_takes():
    """2^27 + 128 columns, 128 deep: the second launch has its own weight scales and its own columns of h and of g and u.
    The weight is one block of rows again and again, with other scales each time."""
    fp8q = require_gpu()
    m, f, k, part = 2, (1 << 27) + 128, 128, 1 << 20
    gen = torch.Generator(device="cuda").manual_seed(3)
    qa, sa = fp8q.fp8_quant_tile(torch.randn((m, k), generator=gen, device="cuda"))
    base, _ = fp8q.fp8_quant_block(torch.randn((part, k), generator=gen, device="cuda") * 0.1)
    qb = torch.empty((2 * f, k), dtype=torch.uint8, device="cuda")
    for r in range(0, 2 * f, part):
        qb[r:r + part] = base[:min(part, 2 * f - r)]
    sb = torch.rand((2 * f // 128, 1), generator=gen, device="cuda") * 1e-3 + 1e-4
    h, gu = fp8q.fp8_gemm_gated(qa, sa, qb, sb, out_dtype=torch.float32, save_gate_up=True)
    dots = (qa.view(torch.float8_e4m3fn).double() * sa.double().t()) @ base.view(torch.float8_e4m3fn).double().t()
    for r in range(0, 2 * f, part):
        n = min(part, 2 * f - r)
        ref = dots[:, :n] * sb[r // 128:(r + n) // 128].double().t().repeat_interleave(128, 1)
        got = gu[:, r:r + n].double()
        assert ((got - ref).norm() / ref.norm()).item() <= 2e-4, r         # the bound of the plain FP8 GEMMs
    for c in range(0, f, 1 << 24):
        g, u = gu[:, c:min(f, c + (1 << 24))].double(), gu[:, f + c:f + min(f, c + (1 << 24))].double()
        ref = g * torch.sigmoid(g) * u
        tol = (18 + 8 * g.abs()) * 2.0 ** -24 * ref.abs() + 2.0 ** -100 * (1 + (g * u).abs())
        assert bool(((h[:, c:c + (1 << 24)].double() - ref).abs() <= tol).all()), c
    del qb, h, gu
    torch.cuda.empty_cache()
