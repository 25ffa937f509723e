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
