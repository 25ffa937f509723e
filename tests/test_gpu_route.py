"""moe_route, moe_route_backward and fp8_moe_dispatch on the GPU against oracle/front.py.

Experts, counts, rows and moved codes are exact.  Tolerances, with u = 2^-24, for a token whose logits lie up to D below
the largest:
  * a term exp2((z - m) log2 e): the difference and the product are one rounding each (relative 2 u of an exponent of up
    to D, so 2 D u of the term), the exponential is good to 2 u: (2 D + 2) u; terms under 2^-126 may be flushed;
  * p: the sum of positive terms (16 per lane, 6 lane steps) has 22 u more than its terms, 1/sum and the product one each:
    (4 D + 30) u; a renormalized weight the same over a sum of up to 32: (8 D + 100) u;
  * sums of p over tokens: one rounding for each of a lane's tokens, of the groups of a workgroup and of the parts that
    meet; all positive;
  * gradient: p's error on p |dp - dot|, and that of dp (dc by its own formula) and of dot (p |dp| summed in 22 steps).
"""

import gc

import numpy as np
import pytest
import torch

from oracle import front as orf
from tests.helpers import assert_bytes_equal, dev, host, require_gpu
from workloads import bf16_bits_as_f32, normal_f32, to_bf16_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -100
F32, BF = torch.float32, torch.bfloat16


def _logits(t, e, dtype, seed, sigma=2.0):
    rng = np.random.default_rng(seed)
    z = normal_f32(rng, (t, e), sigma) + normal_f32(rng, (1, e), 0.7)
    return bf16_bits_as_f32(to_bf16_bits(z)) if dtype == BF else z.astype(np.float32)


def _place(x, dtype):
    """Rows further apart than they are long, NaN in the gaps."""
    rows, cols = x.shape
    per = 16 // torch.empty((), dtype=dtype).element_size()
    buf = torch.full((rows, -(-cols // per) * per + per), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = dev(x).to(dtype)
    return buf[:, :cols]


def _depth(z):
    """How far below the largest a row's finite logits lie (terms beyond 90 are under 2^-126)."""
    m = z.max(axis=1, keepdims=True)
    d = np.where(np.isfinite(z), np.where(np.isfinite(m), m, 0) - z, 0.0)
    return np.minimum(d.max(axis=1, keepdims=True), 90.0)


def _check_route(out, z, k, valid, renormalize):
    weights, experts, counts, loss, slope = out
    w_ref, e_ref, c_ref, l_ref, s_ref = orf.route(z, k, valid, renormalize)
    assert_bytes_equal(host(experts), e_ref, "experts")
    assert host(counts).tolist() == c_ref.tolist()
    depth = _depth(z)
    tol = (8 * depth + 100) * U * w_ref + TINY
    assert np.all(np.abs(host(weights) - w_ref) <= tol)
    assert np.all(np.abs(host(slope) - s_ref) <= 6 * U * s_ref)
    t = z.shape[0]
    steps = -(-t // 4) + 64 + 32 + 16 + 16 + 10             # tokens of a lane, groups, parts, experts
    top = float(depth[valid != 0].max(initial=0.0)) if valid is not None else float(depth.max(initial=0.0))
    assert abs(float(loss) - l_ref) <= (steps + 4 * top + 40) * U * l_ref + TINY


SIZES = [(1, 1, 1), (1, 64, 8), (16, 64, 8), (3, 7, 7), (64, 64, 2), (65, 63, 9), (200, 65, 6), (300, 128, 32), (33, 129, 3),
         (500, 200, 8), (50, 256, 1), (70, 257, 12), (130, 512, 8), (40, 513, 5), (20, 1000, 32), (9, 1024, 32), (1100, 8, 2),
         (700, 100, 8), (300, 1000, 8), (257, 1024, 31), (600, 300, 4)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("t, e, k", SIZES)
def test_moe_route(t, e, k, renormalize, dtype):
    fp8q = require_gpu()
    z = _logits(t, e, dtype, t * 31 + e)
    _check_route(fp8q.moe_route(_place(z, dtype), k, renormalize=renormalize), z.astype(np.float64), k, None, renormalize)


@pytest.mark.parametrize("e, lanes", [(64, 8), (120, 8), (256, 16), (500, 32), (1000, 64)])
@pytest.mark.parametrize("all_lanes, dtype", [(1 << 11, F32), (1 << 12, BF), ((1 << 16) - 64, F32), ((1 << 16) + 64, BF),
                                              ((1 << 17) + 64, F32), ((1 << 18) + 64, BF)])
def test_moe_route_in_workgroups_of_every_size(all_lanes, dtype, e, lanes):
    """One workgroup, several of 256, 512 and 1024 threads, of these in more than one turn; sums by one workgroup and by
    several."""
    fp8q = require_gpu()
    t = all_lanes // lanes
    z = _logits(t, e, dtype, t + e)
    valid = (np.random.default_rng(t).random(t) < 0.9).astype(np.uint8)
    k = 8 if t % 3 else 3
    _check_route(fp8q.moe_route(_place(z, dtype), k, valid=dev(valid)), z.astype(np.float64), k, valid, False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("t, e, k", [(16, 64, 8), (300, 64, 4), (77, 130, 8), (40, 600, 3)])
def test_moe_route_masks(t, e, k, dtype):
    """Tokens that do not count hold NaN; experts taken out by minus infinity, rows with fewer than k left, with one and
    with none; logits at the type's lowest value are logits like others."""
    fp8q = require_gpu()
    rng = np.random.default_rng(5 * t + e)
    z = _logits(t, e, dtype, 9 * t)
    z[:, rng.integers(0, e, 3)] = -np.inf
    z[2] = -np.inf
    z[3, 1:] = -np.inf
    z[4, k // 2:] = -np.inf
    lowest = -float(torch.finfo(dtype).max)
    z[5] = lowest
    z[6, 1::2] = lowest
    valid = (rng.random(t) < 0.7).astype(np.uint8)
    valid[:8] = 1
    valid[7] = 0
    z_in = z.copy()
    z_in[valid == 0] = np.nan
    for mask in (dev(valid), dev(valid).bool()):
        _check_route(fp8q.moe_route(_place(z_in, dtype), k, valid=mask), z.astype(np.float64), k, valid, False)
        _check_route(fp8q.moe_route(_place(z_in, dtype), k, valid=mask, renormalize=True), z.astype(np.float64), k, valid, True)


def test_moe_route_ties_and_zeros():
    """Equal logits go to the lower index, zeros of both signs are equal."""
    fp8q = require_gpu()
    z = np.zeros((4, 100), np.float32)
    z[1, ::2] = -0.0
    z[2, [70, 3, 41]] = 1.0
    z[3] = -5.0
    z[3, [9, 50, 51]] = [1e-40, 3e-40, -1e-40]            # the smallest numbers are in order, too
    _check_route(fp8q.moe_route(dev(z), 6), z.astype(np.float64), 6, None, False)


@pytest.mark.parametrize("e", [9, 64, 100, 250, 500, 1000])
@pytest.mark.parametrize("k", [2, 4, 8, 9])
def test_moe_route_logits_close_to_each_other(e, k):
    """FP32 logits that differ in their last bits alone, among others that do not, of both signs, and FP32 logits that are
    BF16 numbers, of which many are equal: in order, the lower index first."""
    fp8q = require_gpu()
    rng = np.random.default_rng(e + k)
    near = (np.float32(1.5).view(np.int32) + rng.integers(0, 3 * e, (60, e))).astype(np.int32).view(np.float32)
    z = np.concatenate([near, -near, near * np.float32(2.0 ** -140), _logits(60, e, F32, e), _logits(200, e, BF, e)])
    z[5:180:3] += (rng.random((59, e)) < 0.05).astype(np.float32)               # a few above all the others
    z[180:200, ::7] = z[180:200, 1::7][:, :1]                                   # equal ones among those that are not
    _check_route(fp8q.moe_route(_place(z, F32), k, renormalize=True), z.astype(np.float64), k, None, True)
    for rows in (slice(0, 60), slice(240, 440)):                                # waves of one kind alone
        part = np.ascontiguousarray(z[rows])
        _check_route(fp8q.moe_route(_place(part, F32), k), part.astype(np.float64), k, None, False)


@pytest.mark.parametrize("e", [8, 60, 250, 1000])
@pytest.mark.parametrize("k", [4, 5, 6, 7, 8])
def test_moe_route_few_logits_left(e, k):
    """FP32 logits close to each other and not, with all experts, a handful, one and none of them left by minus infinity."""
    fp8q = require_gpu()
    rng = np.random.default_rng(e * k)
    z = np.concatenate([(np.float32(1.5).view(np.int32) + rng.integers(0, 4 * e, (90, e))).astype(np.int32).view(np.float32),
                        _logits(90, e, F32, e + k)])
    z[::7] = -z[::7]
    for i, row in enumerate(z):
        if i % 3:
            row[rng.permutation(e)[i % 10:]] = -np.inf
    _check_route(fp8q.moe_route(_place(z, F32), k, renormalize=True), z.astype(np.float64), k, None, True)


@pytest.mark.parametrize("case", ["no tokens", "none valid", "all minus infinity"])
def test_moe_route_where_no_token_counts(case):
    fp8q = require_gpu()
    t = 0 if case == "no tokens" else 700
    z = torch.randn((t, 16), device="cuda")
    valid = torch.zeros(t, dtype=torch.bool, device="cuda") if case == "none valid" else None
    if case == "all minus infinity":
        z.fill_(-float("inf"))
    w, ex, c, loss, slope = fp8q.moe_route(z, 2, valid=valid, renormalize=True)
    assert not w.any() and bool((ex == -1).all()) and not c.any() and not loss.any() and not slope.any()
    dz = fp8q.moe_route_backward(z, ex, slope, dweights=torch.ones((t, 2), device="cuda"), dloss=torch.ones(1, device="cuda"),
                                 renormalize=True)
    assert dz.shape == (t, 16) and not dz.any()


def test_moe_route_unspecified_logits_stay_in_range():
    """NaN and plus infinity in a token that counts: some expert or none, and the other tokens' rows as they are."""
    fp8q = require_gpu()
    z = _logits(40, 64, F32, 3)
    want = fp8q.moe_route(dev(z), 8)
    z[[3, 9, 20], [1, 2, 63]] = [np.nan, np.inf, np.nan]
    z[30] = np.nan
    w, ex, *_ = fp8q.moe_route(dev(z), 8)
    assert bool(((ex >= -1) & (ex < 64)).all())
    rest = [i for i in range(40) if i not in (3, 9, 20, 30)]
    assert torch.equal(ex[rest], want[1][rest]) and torch.equal(w[rest], want[0][rest])


def _check_backward(dz, z, ex, slope, dw, dloss, renormalize, dtype):
    ref = orf.route_backward(z, ex, slope, dw, dloss, renormalize)
    p = orf.softmax(z)
    depth = _depth(z)
    d_every = abs(dloss) * np.abs(slope)[None, :]
    ok = ex >= 0
    chosen = np.where(ok, np.take_along_axis(p, np.maximum(ex, 0), 1), 0.0)
    total = np.maximum(chosen.sum(axis=1, keepdims=True), 1e-30) if renormalize else 1.0
    a = np.abs(np.where(ok, dw, 0.0))
    size = (a + (a * chosen).sum(axis=1, keepdims=True) / total) / total if renormalize else a      # |dc| with its terms
    size = np.where(ok, size, 0.0)
    dp = np.broadcast_to(d_every, p.shape).copy()
    for j in range(ex.shape[1]):
        np.add.at(dp, (np.arange(len(ex)), np.maximum(ex[:, j], 0)), size[:, j])
    dot = (p * dp).sum(axis=1, keepdims=True)
    rel = (12 * depth + 200) * U                            # p's, twice over a renormalized dc, and the sums' steps
    tol = p * (dp + dot) * rel + TINY
    if dtype == BF:
        tol = tol + np.abs(ref) * 2.0 ** -8
    err = np.abs(dz.double().cpu().numpy() - ref)
    live = ex[:, 0] >= 0
    assert not np.any(err[~live]) and np.all(err[live] <= tol[live]), np.max(err[live] / tol[live])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("t, e, k", SIZES)
def test_moe_route_backward(t, e, k, renormalize, dtype):
    fp8q = require_gpu()
    rng = np.random.default_rng(t + 7 * e)
    z = _logits(t, e, dtype, t * 3 + e)
    if t > 8 and e > 3:                                     # masks: an expert out, a token with one left, one with none
        z[:, 1] = -np.inf
        z[4, 1:] = -np.inf
        z[5] = -np.inf
    valid = (rng.random(t) < 0.8).astype(np.uint8)
    valid[0] = 1
    zd = _place(np.where(valid[:, None] != 0, z, np.nan), dtype)
    _, ex, _, _, slope = fp8q.moe_route(zd, k, valid=dev(valid), renormalize=renormalize)
    dw = normal_f32(rng, (t, k), 1e-3)
    dl = torch.full((1,), 0.013, device="cuda")
    args = (z.astype(np.float64), host(ex), host(slope).astype(np.float64))
    both = fp8q.moe_route_backward(zd, ex, slope, dweights=dev(dw), dloss=dl, renormalize=renormalize)
    _check_backward(both, *args, dw.astype(np.float64), float(dl), renormalize, dtype)
    only_w = fp8q.moe_route_backward(zd, ex, dweights=dev(dw), renormalize=renormalize)
    _check_backward(only_w, *args, dw.astype(np.float64), 0.0, renormalize, dtype)
    only_l = fp8q.moe_route_backward(zd, ex, slope, dloss=dl, renormalize=renormalize)
    _check_backward(only_l, *args, 0.0 * dw.astype(np.float64), float(dl), renormalize, dtype)
    assert not fp8q.moe_route_backward(zd, ex, slope).any()


def test_moe_route_backward_same_expert_twice_and_out_of_range():
    """Choices that moe_route does not make: an expert twice in a token, and indices outside the experts, which are left out."""
    fp8q = require_gpu()
    z = _logits(3, 10, F32, 77)
    ex = np.array([[2, 2, 5], [0, 10, -7], [9, 1 << 30, 9]], np.int32)
    dw = np.array([[1, 2, 3], [4, 5, 6], [7, 8, 9]], np.float32)
    slope = np.linspace(0.1, 1.0, 10).astype(np.float32)
    dl = torch.full((1,), 0.5, device="cuda")
    for renormalize in (False, True):
        ex_ref = np.where((ex >= 0) & (ex < 10), ex, -1)
        ref = orf.route_backward(z, ex_ref, slope, dw, 0.5, renormalize)
        got = fp8q.moe_route_backward(_place(z, F32), dev(ex), dev(slope), dweights=dev(dw), dloss=dl, renormalize=renormalize)
        assert np.all(np.abs(host(got) - ref) <= 500 * U * 40)      # terms up to 40 in size


# ---------------------------------------------------------------------------
# fp8_moe_dispatch
# ---------------------------------------------------------------------------
def _check_dispatch(fp8q, experts, e, d, seed, extra=0):
    rng = np.random.default_rng(seed)
    t, k = experts.shape
    q = rng.integers(0, 256, (t, d)).astype(np.uint8)
    s = rng.random((d // 128, t)).astype(np.float32) + np.float32(0.5)
    rows = fp8q.moe_max_rows(t, k, e) + extra
    buf = torch.full((rows + 2, d + 32), 0x33, dtype=torch.uint8, device="cuda")
    a, sa = buf[1:rows + 1, :d], torch.full((d // 128, rows), -3.0, device="cuda")
    qd = torch.full((t, d + 16), 0x77, dtype=torch.uint8, device="cuda")[:, :d]
    qd.copy_(dev(q))
    got = fp8q.fp8_moe_dispatch(dev(experts), qd, dev(s), e, a=a, a_scales=sa)
    group, row_of_slot, token_of_row = orf.dispatch(experts, e, rows)
    assert_bytes_equal(host(got[2]), group, "group_of_mtile")
    assert_bytes_equal(host(got[3]), row_of_slot, "row_of_slot")
    assert_bytes_equal(host(got[4]), token_of_row, "token_of_row")
    used = np.repeat(group >= 0, 128)
    want_a = np.where(used[:, None], 0, 0x33).astype(np.uint8) * np.ones((1, d), np.uint8)
    want_s = np.broadcast_to(np.where(used, np.float32(2.0 ** -126), np.float32(-3.0))[None, :], (d // 128, rows)).copy()
    live = token_of_row >= 0
    want_a[live] = q[token_of_row[live]]
    want_s[:, live] = s[:, token_of_row[live]]
    assert_bytes_equal(host(a), want_a, "codes")
    assert_bytes_equal(host(sa), want_s, "scales")
    buf[1:rows + 1, :d] = 0x33
    assert bool((buf == 0x33).all()), "written outside the output"


@pytest.mark.parametrize("t, k, e, d", [(1, 1, 1, 128), (1, 8, 64, 1152), (16, 8, 64, 256), (37, 3, 5, 1024), (300, 2, 7, 384), (1024, 8, 64, 128),
                                        (1023, 8, 200, 128), (1025, 8, 64, 128), (2500, 4, 1000, 128), (900, 32, 33, 128),
                                        (5000, 2, 3, 256), (1, 32, 1024, 2176), (9000, 1, 1, 128), (1024, 1, 3, 1152),
                                        (1025, 1, 3, 1152), (512, 2, 1024, 128), (33, 31, 1, 2048),
                                        (4096, 1, 7, 1152), (1366, 3, 9, 128), (2048, 2, 1000, 256), (8192, 1, 64, 128)])
def test_dispatch(t, k, e, d):
    fp8q = require_gpu()
    rng = np.random.default_rng(t + e)
    p = np.arange(1, e + 1) ** -1.1
    experts = rng.choice(e, size=(t, k), p=p / p.sum()).astype(np.int32)       # an expert may come twice in a token
    _check_dispatch(fp8q, experts, e, d, seed=t, extra=128 * (t % 3))


@pytest.mark.parametrize("t, k", [(100, 8), (200, 8), (600, 8), (3000, 8)])
def test_dispatch_choices_outside_the_experts(t, k):
    """-1, and anything else outside the range, gets no row; an expert without rows no tile."""
    fp8q = require_gpu()
    rng = np.random.default_rng(t)
    experts = rng.integers(0, 20, (t, k)).astype(np.int32)
    experts[rng.random((t, k)) < 0.4] = -1
    experts[experts == 7] = 20
    experts[0, 0], experts[1, 1] = 1 << 30, -(1 << 31)
    _check_dispatch(fp8q, experts, 20, 256, seed=3)
    _check_dispatch(fp8q, np.full((t, k), -1, np.int32), 20, 256, seed=4)


@pytest.mark.parametrize("counts", [[128, 128], [129, 0, 127], [0, 0, 256], [1, 1, 1, 1], [128 * 70, 1]])
def test_dispatch_at_tile_edges(counts):
    fp8q = require_gpu()
    experts = np.concatenate([np.full(c, e, np.int32) for e, c in enumerate(counts)])
    experts = np.random.default_rng(1).permutation(experts)[:, None].copy()
    _check_dispatch(fp8q, experts, len(counts), 256, seed=6)


@pytest.mark.parametrize("t", [40, 300, 9000])
def test_dispatch_into_outputs_of_the_callers(t):
    """Any of them given alone says how many rows there are; FP8 tensors are codes as bytes are."""
    fp8q = require_gpu()
    rng = np.random.default_rng(t)
    ex = dev(rng.integers(-1, 9, (t, 4)).astype(np.int32))
    q, s = fp8q.fp8_rmsnorm(torch.randn((t, 256), device="cuda"), torch.ones(256, device="cuda"))
    rows = fp8q.moe_max_rows(t, 4, 9) + 256
    i = lambda *sh: torch.full(sh, 99, dtype=torch.int32, device="cuda")       # noqa: E731
    want = orf.dispatch(host(ex), 9, rows)
    live = torch.from_numpy(want[2] >= 0).cuda()
    of = dev(want[2]).long()[live]
    for kw in (dict(a=torch.zeros((rows, 256), device="cuda").to(torch.float8_e4m3fn)),
               dict(a_scales=torch.zeros((2, rows), device="cuda")), dict(group_of_mtile=i(rows // 128)),
               dict(token_of_row=i(rows)), dict(token_of_row=i(rows), row_of_slot=i(t, 4))):
        got = fp8q.fp8_moe_dispatch(ex, q.view(torch.float8_e4m3fn), s, 9, **kw)
        for name, t_ in kw.items():
            at = ("a", "a_scales", "group_of_mtile", "row_of_slot", "token_of_row").index(name)
            assert got[at].data_ptr() == t_.data_ptr()
        for g, w in zip(got[2:], want):
            assert_bytes_equal(host(g), w, "maps")
        assert torch.equal(got[0].view(torch.uint8)[live], q[of]) and torch.equal(got[1][:, live], s[:, of])


def test_dispatch_empty():
    fp8q = require_gpu()
    e8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")           # noqa: E731
    a, sa, g, r, tr = fp8q.fp8_moe_dispatch(torch.empty((0, 2), dtype=torch.int32, device="cuda"), e8(0, 256),
                                            torch.empty((2, 0), device="cuda"), 8)
    assert a.shape == (0, 256) and g.shape == (0,) and r.shape == (0, 2) and tr.shape == (0,)
    # room for tiles and no tokens: the maps say so
    a, sa, g, r, tr = fp8q.fp8_moe_dispatch(torch.empty((0, 2), dtype=torch.int32, device="cuda"), e8(0, 256),
                                            torch.empty((2, 0), device="cuda"), 8, a=e8(256, 256))
    assert bool((g == -1).all()) and bool((tr == -1).all()) and g.shape == (2,)
    # no columns: the maps alone
    ex = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    a, sa, g, r, tr = fp8q.fp8_moe_dispatch(ex, e8(1, 0), torch.empty((0, 1), device="cuda"), 2)
    assert g.tolist() == [0, 1] and r.tolist() == [[128, 0]] and int(tr[0]) == int(tr[128]) == 0 and int((tr >= 0).sum()) == 2


def test_route_and_dispatch_refusals():
    fp8q = require_gpu()
    f = lambda *s: torch.zeros(s, device="cuda")                               # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")            # noqa: E731
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")            # noqa: E731
    with pytest.raises(TypeError, match="logits must be"):
        fp8q.moe_route(f(4, 8).half(), 2)
    with pytest.raises(ValueError, match="valid has shape"):
        fp8q.moe_route(f(4, 8), 2, valid=u(5))
    with pytest.raises(TypeError, match="valid must be"):
        fp8q.moe_route(f(4, 8), 2, valid=i(4))
    with pytest.raises(TypeError, match="experts must be"):
        fp8q.moe_route(f(4, 8), 2, experts=torch.zeros((4, 2), dtype=torch.int64, device="cuda"))
    for k, status in ((0, fp8q.ERR_UNSUPPORTED), (9, fp8q.ERR_SHAPE), (-1, fp8q.ERR_SHAPE)):
        with pytest.raises(fp8q.Fp8qError) as err:
            fp8q.moe_route(f(4, 8), k)
        assert err.value.status == status
    with pytest.raises(fp8q.Fp8qError) as err:
        fp8q.moe_route(f(4, 1028), 2)
    assert err.value.status == fp8q.ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="dloss goes by slope"):
        fp8q.moe_route_backward(f(4, 8), i(4, 2), dloss=f(1))
    with pytest.raises(ValueError, match="dweights has shape"):
        fp8q.moe_route_backward(f(4, 8), i(4, 2), dweights=f(4, 3))
    with pytest.raises(ValueError, match="experts has shape"):
        fp8q.moe_route_backward(f(4, 8), i(5, 2))
    with pytest.raises(ValueError, match="T..k. tensor"):
        fp8q.moe_route_backward(f(4, 8), i(4))
    with pytest.raises(TypeError, match="dlogits must be"):
        fp8q.moe_route_backward(f(4, 8), i(4, 2), dlogits=f(4, 8).to(BF))
    with pytest.raises(ValueError, match="scales has shape"):
        fp8q.fp8_moe_dispatch(i(4, 2), u(4, 128), f(4, 1), 8)
    with pytest.raises(TypeError, match="experts must be"):
        fp8q.fp8_moe_dispatch(i(4, 2).long(), u(4, 128), f(1, 4), 8)
    with pytest.raises(ValueError, match="no such sizes"):
        fp8q.fp8_moe_dispatch(i(4, 2), u(4, 128), f(1, 4), 0)
    with pytest.raises(ValueError, match="a_scales has shape"):
        fp8q.fp8_moe_dispatch(i(4, 2), u(4, 128), f(1, 4), 8, a=u(1024, 128), a_scales=f(1, 128))
    with pytest.raises(fp8q.Fp8qError) as err:                                 # too few rows for 8 slots of 8 experts
        fp8q.fp8_moe_dispatch(i(4, 2), u(4, 128), f(1, 4), 8, a=u(896, 128))
    assert err.value.status == fp8q.ERR_SHAPE


def test_route_refuses_more_experts_than_memory_holds():
    fp8q = require_gpu()
    for k in (300, 1 << 40):
        with pytest.raises(fp8q.Fp8qError) as err:
            fp8q.moe_route(torch.zeros((4, 8), device="cuda"), k)
        assert err.value.status == fp8q.ERR_SHAPE


@pytest.mark.parametrize("e, k", [(64, 65), (64, 200), (64, 255), (64, 40), (8, 9), (1024, 33), (1032, 8)])
@pytest.mark.parametrize("given", [False, True])
def test_route_refuses_before_memory_is_asked_for(e, k, given):
    """The native call (no output given) and the other one alike: more places than there are experts or than are
    supported, more experts than are."""
    fp8q = require_gpu()
    t = 1 << 16
    z = torch.zeros((t, e), dtype=BF, device="cuda")
    kw = dict(loss=torch.zeros(1, device="cuda")) if given else {}
    torch.cuda.synchronize()
    gc.collect()                                   # tensors of other tests that an exception's frames held
    torch.cuda.reset_peak_memory_stats()
    peak = torch.cuda.max_memory_allocated()
    with pytest.raises(fp8q.Fp8qError) as err:
        fp8q.moe_route(z, k, **kw)
    assert err.value.status == (fp8q.ERR_SHAPE if k > e else fp8q.ERR_UNSUPPORTED)
    assert torch.cuda.max_memory_allocated() == peak
