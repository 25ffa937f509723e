"""The operators in front of the projections together, as a layer of experts uses them: norm with the residual, routing by
the normed tokens, dispatch of their codes, the grouped product; and back through the routing and the norm.  On streams of
the caller's, captured into a HIP graph, from two threads, and through the native call path and ctypes alike."""

import threading

import numpy as np
import pytest
import torch

from oracle import front as orf, gemm as og
from tests.helpers import dev_bf16, host, require_gpu
from tests.test_gpu_output_streams import _owner
from workloads import normal_f32, to_bf16_bits

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
E, K_CHOSEN = 6, 2


def _inputs(seed, t, d=256, f=128):
    rng = np.random.default_rng(seed)
    r = lambda *s, sigma=1.0: dev_bf16(to_bf16_bits(normal_f32(rng, s, sigma)))              # noqa: E731
    valid = torch.from_numpy((rng.random(t) < 0.9).astype(np.uint8)).cuda()
    return (r(t, d), r(t, d, sigma=2.0), 1.0 + r(1, d, sigma=0.2)[0], r(E + -E % 8, d, sigma=0.1), r(E * f, d, sigma=0.05),
            r(t, d, sigma=1e-3), r(t, d, sigma=1e-3), valid)


def _logits(y, wr):
    # the product on the current stream; E columns of wider rows
    return (y @ wr.t())[:, :E]


def _layer(fp8q, x, res, w, wr, we, dy, dh, valid, stream=None, logits=None):
    """Forward and back; every output."""
    q, s, h, rstd, y = fp8q.fp8_rmsnorm(x, w, residual=res, save_rstd=True, save_y=True, stream=stream)
    z = _logits(y, wr) if logits is None else logits
    weights, experts, counts, loss, slope = fp8q.moe_route(z, K_CHOSEN, valid=valid, renormalize=True, stream=stream)
    rows = fp8q.moe_max_rows(x.shape[0], K_CHOSEN, E)
    a = torch.zeros((rows, x.shape[1]), dtype=torch.uint8, device="cuda") if stream is None else None
    sa = torch.zeros((x.shape[1] // 128, rows), device="cuda") if stream is None else None
    a, sa, gmap, slots, tokens = fp8q.fp8_moe_dispatch(experts, q, s, E, a=a, a_scales=sa, stream=stream)
    qw, sw = fp8q.fp8_quant_block(we, stream=stream)
    f = we.shape[0] // E
    c = torch.zeros((rows, f), dtype=BF, device="cuda") if stream is None else None
    c = fp8q.fp8_gemm_blockscaled_grouped(gmap, a, sa, qw.view(E, f, -1), sw.view(E, f // 128, -1), c=c, stream=stream)
    dz = fp8q.moe_route_backward(z, experts, slope, dweights=weights, dloss=loss, renormalize=True, stream=stream)
    dx, dw = fp8q.rmsnorm_backward(dy, h, w, rstd, dh=dh, stream=stream)
    dual = fp8q.fp8_rmsnorm(x, w, residual=res, transposed=True, stream=stream)
    i8 = fp8q.int8_rmsnorm(h, w, stream=stream)
    return [q, s, h, rstd, y, weights, experts, counts, loss, slope, gmap, slots, tokens, c, dz, dx, dw, *dual, *i8, a, sa]


def _bytes(t):
    return host(t.contiguous().view(torch.uint8))


def _same(got, want, used=None):
    for i, (x, y) in enumerate(zip(got, want)):
        assert np.array_equal(_bytes(x), y), i


def test_layer_of_experts():
    """Each expert's product has, row for row, what the oracle's product of the dispatched codes has; a token's rows hold
    the token's own codes."""
    fp8q = require_gpu()
    args = _inputs(3, 300)
    out = _layer(fp8q, *args)
    q, s, weights, experts, gmap, slots, tokens, c, a, sa = (out[i] for i in (0, 1, 5, 6, 10, 11, 12, 13, -2, -1))
    group, rows, toks = orf.dispatch(host(experts), E, a.shape[0])
    assert np.array_equal(host(gmap), group) and np.array_equal(host(slots), rows) and np.array_equal(host(tokens), toks)
    live = toks >= 0
    assert np.array_equal(host(a)[live], host(q)[toks[live]]) and not host(a)[~live].any()
    qw, sw = fp8q.fp8_quant_block(args[4])
    f = args[4].shape[0] // E
    ref = og.grouped_ref(host(a), host(sa), host(qw).reshape(E, f, -1), host(sw).reshape(E, f // 128, -1), np.maximum(group, 0))
    got = c.double().cpu().numpy()
    assert og.rel_frobenius(got[live], og.round_bf16(ref)[live]) <= 1e-3 and not got[~live].any()
    valid = host(args[-1])
    assert np.all((host(experts) >= 0) == (valid[:, None] != 0)) and float(out[8][0]) > 0.9


@pytest.mark.parametrize("t", [1, 300])
def test_layer_on_a_user_stream(t):
    fp8q = require_gpu()
    args = _inputs(31, t)
    want = [_bytes(x) for x in _layer(fp8q, *args)]
    busy = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):                                    # the default stream is busy meanwhile
        busy = busy @ busy.t() * 1e-3
    with torch.cuda.stream(s):
        got = _layer(fp8q, *args)
    s.synchronize()
    _same(got, want)


@pytest.mark.parametrize("t", [2, 300])
def test_layer_on_a_stream_argument_alone(t):
    """stream=s from the default stream, whose own allocations and work go on meanwhile: workspaces and intermediate
    tensors are dropped as soon as the next call is made."""
    fp8q = require_gpu()
    args = _inputs(61, t)
    first = _layer(fp8q, *args)
    z = _logits(first[4], args[3]).contiguous()
    z = torch.nn.functional.pad(z, (0, -E % 4))[:, :E]
    want = [_bytes(x) for x in first[:13] + first[14:-2]]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = _layer(fp8q, *args, stream=s, logits=z)
        noise = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 18)]
        s.synchronize()
        for i, (x, y) in enumerate(zip(got[:13] + got[14:-2], want)):
            if i != 14 - 1:                               # the logits' gradient: of the BF16 logits padded anew
                assert np.array_equal(_bytes(x), y), i
        assert all(bool((x == 0x55).all()) for x in noise)


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("t", [2, 300, 5000])
def test_logits_gradient_on_a_stream_argument_alone(t, given, form):
    """moe_route_backward with stream=s behind work of s that writes what it reads, into new and given outputs: the logits of
    the layer with rows padded to 16 bytes, as the default stream gives it for them."""
    fp8q = require_gpu()
    args = _inputs(61, t)
    layer = _layer(fp8q, *args)
    z = torch.nn.functional.pad(_logits(layer[4], args[3]).contiguous(), (0, 2))[:, :E]
    weights, experts, loss, slope = (layer[i] for i in (5, 6, 8, 9))
    want = _bytes(fp8q.moe_route_backward(z, experts, slope, dweights=weights, dloss=loss, renormalize=True))
    assert np.array_equal(want, _bytes(layer[14]))        # the layer's own logits lie in rows of 8
    s = torch.cuda.Stream()
    late = [torch.zeros_like(x) for x in (weights, slope, loss)]
    zl, el = torch.zeros((t, 8), dtype=BF, device="cuda")[:, :E], torch.full_like(experts, -1)
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        for x in (zl, *late):
            x.zero_()
        out = torch.full((t, 8), 7.0, dtype=BF, device="cuda")[:, :E] if given else None
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(4):
                busy = busy @ busy.t() * 1e-3
            for x, y in zip((zl, el, *late), (z, experts, weights, slope, loss)):
                x.copy_(y)
        dz = fp8q.moe_route_backward(zl, el, late[1], dweights=late[0], dloss=late[2], renormalize=True, dlogits=out,
                                     stream=s if form == "stream" else s.cuda_stream)
        noise = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 18)]
        s.synchronize()
        assert np.array_equal(_bytes(dz), want) and (not given or dz is out)
        assert all(bool((x == 0x55).all()) for x in noise)


@pytest.mark.parametrize("t", [1, 300, 5000])
def test_layer_captured_in_a_hip_graph_and_replayed(t):
    """Two graphs of the layer on buffers of their own, replayed in turn with new inputs and eager work between: each has
    workspaces of its own (5000 tokens: more slots than one workgroup plans)."""
    fp8q = require_gpu()
    graphs = []
    for n in range(2):
        bufs = _inputs(41 + n, t)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _layer(fp8q, *bufs)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _layer(fp8q, *bufs)
        torch.cuda.synchronize()
        graphs.append((graph, bufs, out))
    for seed in (51, 52, 53):
        for n, (graph, bufs, out) in enumerate(graphs):
            args = _inputs(seed + 10 * n, t)
            want = [_bytes(x) for x in _layer(fp8q, *args)]
            for b, x in zip(bufs, args):
                b.copy_(x)
            graph.replay()
            torch.cuda.synchronize()
            for i, (x, y) in enumerate(zip(out[:13] + out[14:-2], want[:13] + want[14:-2])):
                assert np.array_equal(_bytes(x), y), (seed, n, i)
            live = host(out[12]) >= 0                     # rows of a tile that is not in use keep what they hold
            assert np.array_equal(host(out[13].float())[live], host(_layer(fp8q, *args)[13].float())[live])


def test_two_threads_at_once():
    """Calls from two threads on streams of their own do not share anything."""
    fp8q = require_gpu()
    args = [_inputs(71, 300), _inputs(72, 700)]
    want = [[_bytes(x) for x in _layer(fp8q, *a)] for a in args]
    failed = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                with torch.cuda.stream(s):
                    got = _layer(fp8q, *args[i])
                s.synchronize()
                with torch.cuda.stream(s):
                    _same(got, want[i])
        except BaseException as e:                        # noqa: B902 (told to the main thread)
            failed.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_native_and_ctypes_calls_agree(monkeypatch):
    """The native call path takes the usual calls and answers what the ctypes path does, for every option."""
    fp8q = require_gpu()
    from precision_fp8_quant_amd import front
    assert front._native is not None
    x, res, w, _, _, dy, dh, valid = _inputs(81, 37)
    odd = torch.randn(9, 336, device="cuda")[:, :333]
    wo = torch.rand(333, device="cuda") + 0.5
    z = torch.randn(37, 64, device="cuda")
    rstd = torch.rand(37, device="cuda") + 0.5
    q, s = fp8q.fp8_rmsnorm(x, w)
    _, ex, _, _, slope = fp8q.moe_route(z, 5)
    dwt, dl = torch.randn(37, 5, device="cuda"), torch.full((1,), 0.3, device="cuda")
    rows = fp8q.moe_max_rows(37, 5, 64)
    a, sa = torch.zeros((rows, 256), dtype=torch.uint8, device="cuda"), torch.zeros((2, rows), device="cuda")
    calls = [("fp8_rmsnorm", (x, w), {}), ("fp8_rmsnorm", (x, w.float()), dict(residual=res, mode=fp8q.POW2, save_rstd=True)),
             ("fp8_rmsnorm", (x, w), dict(residual=res, transposed=True, save_rstd=True, save_y=True)),
             ("fp8_rmsnorm", (x, w), dict(transposed=True, eps=0.5)), ("fp8_rmsnorm", (x[:1], w), dict(save_y=True)),
             ("int8_rmsnorm", (odd, wo), {}), ("int8_rmsnorm", (odd, wo), dict(residual=odd, save_rstd=True, save_y=True)),
             ("int8_rmsnorm", (x, w), dict(residual=res)), ("rmsnorm_backward", (dy, x, w, rstd), {}),
             ("rmsnorm_backward", (dy, x, w, rstd), dict(dh=dh)), ("rmsnorm_backward", (odd, odd, wo, rstd[:9].clone()), {}),
             ("moe_route", (z, 5), {}), ("moe_route", (z, 8), dict(valid=valid, renormalize=True)),
             ("moe_route", (z.to(BF), 3), dict(valid=valid.bool())),
             ("moe_route_backward", (z, ex, slope), dict(dweights=dwt, dloss=dl, renormalize=True)),
             ("moe_route_backward", (z, ex), dict(dweights=dwt)), ("moe_route_backward", (z.to(BF), ex, slope), dict(dloss=dl)),
             ("fp8_moe_dispatch", (ex, q, s, 64), dict(a=a, a_scales=sa)), ("fp8_moe_dispatch", (ex, q, s, 64), {})]
    seen = []

    class Native:
        def __getattr__(self, name):
            real = getattr(native, name)

            def call(*args):
                r = real(*args)
                seen.append(r is not None)
                return r
            return call

    native = front._native
    for name, args, kw in calls:
        monkeypatch.setattr(front, "_native", Native())
        got = getattr(fp8q, name)(*args, **kw)
        monkeypatch.setattr(front, "_native", None)
        want = getattr(fp8q, name)(*args, **kw)
        got, want = [g if isinstance(g, tuple) else (g,) for g in (got, want)]
        assert len(got) == len(want), name
        for i, (g, t) in enumerate(zip(got, want)):
            assert g.shape == t.shape and g.dtype == t.dtype and g.stride() == t.stride(), (name, i)
            if name == "fp8_moe_dispatch" and i < 2 and not kw:           # rows that are not in use hold anything
                continue
            assert torch.equal(g.view(torch.uint8) if g.is_contiguous() else g, t.view(torch.uint8) if t.is_contiguous() else t), (name, i)
    assert seen == [True] * len(calls)


@pytest.mark.parametrize("form", ["stream", "handle"])
def test_new_outputs_belong_to_the_given_stream(form):
    """As for the package's other calls: the allocator reuses a block in the order of the stream that it was allocated on."""
    fp8q = require_gpu()
    x, res, w, _, _, dy, dh, valid = _inputs(91, 130)
    z = torch.randn(130, 64, device="cuda")
    q, s = fp8q.fp8_rmsnorm(x, w)
    rstd = torch.rand(130, device="cuda")
    _, ex, _, _, slope = fp8q.moe_route(z, 5)
    torch.cuda.synchronize()
    calls = [lambda st: fp8q.fp8_rmsnorm(x, w, residual=res, transposed=True, save_rstd=True, save_y=True, stream=st),
             lambda st: fp8q.int8_rmsnorm(x, w, residual=res, save_rstd=True, save_y=True, stream=st),
             lambda st: fp8q.rmsnorm_backward(dy, x, w, rstd, dh=dh, stream=st),
             lambda st: fp8q.moe_route(z, 5, valid=valid, stream=st),
             lambda st: [fp8q.moe_route_backward(z, ex, slope, dloss=torch.ones(1, device="cuda"), stream=st)],
             lambda st: fp8q.fp8_moe_dispatch(ex, q, s, 64, stream=st)]
    for i, call in enumerate(calls):
        s2 = torch.cuda.Stream()
        assert all(_owner(t) == torch.cuda.current_stream().cuda_stream for t in call(None)), i
        torch.cuda.synchronize()
        before = torch.cuda.current_stream()
        got = call(s2 if form == "stream" else s2.cuda_stream)
        assert torch.cuda.current_stream() == before
        s2.synchronize()
        assert all(_owner(t) == s2.cuda_stream for t in got), i
