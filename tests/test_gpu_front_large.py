"""Operators in front of the projections on tensors beyond 2^31 elements or bytes: what they give for rows past the limit is
what a call on those rows alone gives.  Inputs are drawn on the GPU (seeded)."""

import pytest
import torch

from tests.helpers import require_gpu
from workloads import device_fp8_codes, device_normal_bf16

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _w(d):
    return 1.0 + 0.2 * torch.randn(d, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")


def test_norm_beyond_2g_elements():
    """270336 x 8192 BF16 (2.2e9 elements), both tilings and the single one, and the gradient."""
    fp8q = require_gpu()
    m, d, lo = 270336, 8192, 270336 - 256
    x, w = device_normal_bf16(1, (m, d)), _w(d)
    q, s, qt, st, rstd, y = fp8q.fp8_rmsnorm(x, w, transposed=True, save_rstd=True, save_y=True)
    one = fp8q.fp8_rmsnorm(x[lo:].clone(), w, transposed=True, save_rstd=True, save_y=True)
    assert torch.equal(q[lo:], one[0]) and torch.equal(s[:, lo:], one[1]) and torch.equal(qt[:, lo:], one[2])
    assert torch.equal(st[lo // 128:], one[3]) and torch.equal(rstd[lo:], one[4]) and torch.equal(y[lo:], one[5])
    del q, s, qt, st
    q, s = fp8q.fp8_rmsnorm(x, w)
    assert torch.equal(q[lo:], one[0]) and torch.equal(s[:, lo:], one[1])
    q, s = fp8q.int8_rmsnorm(x, w)
    i1 = fp8q.int8_rmsnorm(x[lo:].clone(), w)
    assert torch.equal(q[lo:], i1[0]) and torch.equal(s[lo:], i1[1])
    del q, s
    dx, dw = fp8q.rmsnorm_backward(y, x, w, rstd, dh=x)
    d1, _ = fp8q.rmsnorm_backward(y[lo:].clone(), x[lo:].clone(), w, rstd[lo:].clone(), dh=x[lo:].clone())
    assert torch.equal(dx[lo:], d1)
    # dw = sum y xhat: positive where the weight is, about m times the weight
    assert float((dw / w / m - 1).abs().max()) < 0.05
    del x, y, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_route_beyond_2g_elements(dtype):
    """2.2e6 x 1000 logits (2.2e9 elements)."""
    fp8q = require_gpu()
    t, e, k, lo = 2_200_000, 1000, 4, 2_200_000 - 999
    z = torch.empty((t, e), dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    w, ex, counts, loss, slope = fp8q.moe_route(z, k)
    w1, ex1, *_ = fp8q.moe_route(z[lo:].clone(), k)
    assert torch.equal(w[lo:], w1) and torch.equal(ex[lo:], ex1) and int(counts.sum()) == t * k
    top = z[lo:].float().topk(k, 1)
    assert torch.equal(top.values, z[lo:].float().gather(1, ex[lo:].long()))
    assert abs(float(loss) - 1.0) < 0.01                  # all experts alike: even shares
    dl, dw = torch.ones(1, device="cuda"), torch.randn(t, k, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    dz = fp8q.moe_route_backward(z, ex, slope, dweights=dw, dloss=dl)
    d1 = fp8q.moe_route_backward(z[lo:].clone(), ex[lo:].clone(), slope, dweights=dw[lo:].clone(), dloss=dl)
    assert torch.equal(dz[lo:], d1)
    del z, dz
    torch.cuda.empty_cache()


def test_dispatch_beyond_2g_bytes():
    """40000 tokens of 8 experts, 7168 channels: 2.3e9 bytes of rows."""
    fp8q = require_gpu()
    t, k, e, d = 40000, 8, 64, 7168
    q = device_fp8_codes(4, (t, d))
    s = torch.rand((d // 128, t), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda") + 0.5
    z = torch.randn((t, e), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    ex = fp8q.moe_route(z, k)[1]
    a, sa, gmap, slots, tokens = fp8q.fp8_moe_dispatch(ex, q, s, e)
    assert int((tokens >= 0).sum()) == t * k and bool((slots >= 0).all())
    flat = slots.view(-1).long()
    assert torch.equal(tokens[flat], torch.arange(t, device="cuda", dtype=torch.int32).repeat_interleave(k))
    assert torch.equal(gmap[flat // 128], ex.view(-1))
    order = torch.sort(ex.view(-1), stable=True).indices  # rows of an expert in the order of their slots
    assert bool((flat[order].diff()[ex.view(-1)[order].diff() == 0] == 1).all())
    far = tokens.nonzero().view(-1)
    far = torch.cat([(tokens >= 0).nonzero().view(-1)[-2000:], (tokens >= 0).nonzero().view(-1)[:100]])
    assert int(far.max()) * d > 1 << 31
    assert torch.equal(a[far], q[tokens[far].long()]) and torch.equal(sa[:, far], s[:, tokens[far].long()])
    pads = ((tokens < 0) & (gmap.repeat_interleave(128) >= 0)).nonzero().view(-1)
    assert not a[pads].any() and bool((sa[:, pads] == 2.0 ** -126).all())
    del a, q
    torch.cuda.empty_cache()
