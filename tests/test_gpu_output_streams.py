"""Outputs that a call allocates belong to the stream that the call goes to: torch's allocator reuses a block in the
order of the stream that it was allocated on, so any other owner would let a freed output be handed out while the
kernel still writes it."""

import pytest
import torch

from tests.helpers import require_gpu
from tests.test_gpu_ffn import _chain, _chain_inputs

pytestmark = pytest.mark.gpu

BF, I8 = torch.bfloat16, torch.int8


def _calls(fp8q):
    """Every entry point with all of its outputs allocated, by name: a function of the stream."""
    x = torch.randn(256, 384, device="cuda", dtype=BF)
    w = torch.randn(512, 384, device="cuda", dtype=BF)
    qx, sx = fp8q.fp8_quant_tile(x)
    qw, sw = fp8q.fp8_quant_block(w)
    gmap = torch.zeros(2, dtype=torch.int32, device="cuda")
    dh, gu = torch.randn(130, 256, device="cuda"), torch.randn(130, 512, device="cuda")
    odd = torch.randn(9, 336, device="cuda")[:, :333]
    ia, isa = fp8q.int8_quant_rows(odd)
    ib, isb = fp8q.int8_quant_rows(torch.randn(70, 336, device="cuda")[:, :333])
    torch.cuda.synchronize()
    return {
        "fp8_quant_tile": lambda s: fp8q.fp8_quant_tile(x, stream=s),
        "fp8_quant_tile_dual": lambda s: fp8q.fp8_quant_tile_dual(x, stream=s),
        "fp8_quant_block": lambda s: fp8q.fp8_quant_block(w, transposed=True, stream=s),
        "fp8_gemm_blockscaled": lambda s: [fp8q.fp8_gemm_blockscaled(fp8q.FPROP, qx, sx, qw, sw, stream=s)],
        "fp8_gemm_blockscaled_grouped": lambda s: [fp8q.fp8_gemm_blockscaled_grouped(
            gmap, qx, sx, qw.unsqueeze(0), sw.unsqueeze(0), stream=s)],
        "fp8_requant_1x128_to_128x1": lambda s: fp8q.fp8_requant_1x128_to_128x1(qx, sx, stream=s),
        "fp8_gemm_gated": lambda s: fp8q.fp8_gemm_gated(qx, sx, qw, sw, save_gate_up=True, stream=s),
        "fp8_gated_backward": lambda s: fp8q.fp8_gated_backward(dh, gu, stream=s),
        "int8_quant_rows": lambda s: fp8q.int8_quant_rows(odd, stream=s),
        "int8_gemm": lambda s: [fp8q.int8_gemm(ia, isa, ib, isb, stream=s)],
        "int8_gemm_gated": lambda s: [fp8q.int8_gemm_gated(ia, isa, ib, isb, stream=s)],
    }


NAMES = ["fp8_quant_tile", "fp8_quant_tile_dual", "fp8_quant_block", "fp8_gemm_blockscaled",
         "fp8_gemm_blockscaled_grouped", "fp8_requant_1x128_to_128x1", "fp8_gemm_gated", "fp8_gated_backward",
         "int8_quant_rows", "int8_gemm", "int8_gemm_gated"]


def _owner(t):
    """Handle of the stream whose pool holds t's block."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any segment of the allocator")


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_new_outputs_belong_to_the_given_stream(name, form):
    fp8q = require_gpu()
    call = _calls(fp8q)[name]
    s = torch.cuda.Stream()
    want = call(None)
    assert all(_owner(t) == torch.cuda.current_stream().cuda_stream for t in want)
    torch.cuda.synchronize()
    before = torch.cuda.current_stream()
    got = call(s if form == "stream" else s.cuda_stream)
    assert torch.cuda.current_stream() == before
    s.synchronize()
    assert all(_owner(t) == s.cuda_stream for t in got)
    assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(got, want))


def test_given_outputs_leave_the_current_stream_alone(monkeypatch):
    """Where nothing is allocated, a call on another stream does not change the current one on the way."""
    fp8q = require_gpu()
    x, w = torch.randn(256, 384, device="cuda", dtype=BF), torch.randn(512, 384, device="cuda", dtype=BF)
    args = dict(zip("q scales q_t scales_t".split(), fp8q.fp8_quant_tile_dual(x)))
    qw, sw = fp8q.fp8_quant_block(w)
    h, gu = fp8q.fp8_gemm_gated(args["q"], args["scales"], qw, sw, save_gate_up=True)
    back = dict(zip("q scales q_t scales_t".split(), fp8q.fp8_gated_backward(h, gu)))
    want = [t.clone() for t in (h, gu, *back.values())]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    monkeypatch.setattr(torch.cuda, "stream", None)
    fp8q.fp8_quant_tile_dual(x, **args, stream=s)
    fp8q.fp8_gemm_gated(args["q"], args["scales"], qw, sw, h=h, gu=gu, stream=s)
    fp8q.fp8_gated_backward(h, gu, **back, stream=s)
    q, sq = torch.empty(256, 384, device="cuda", dtype=I8), torch.empty(256, device="cuda")
    fp8q.int8_quant_rows(x, q=q, scales=sq, stream=s)
    fp8q.int8_gemm(q, sq, q, sq, c=torch.empty(256, 256, device="cuda"), stream=s)
    fp8q.int8_gemm_gated(q, sq, q, sq, h=torch.empty(256, 128, device="cuda"), stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((h, gu, *back.values()), want))


def test_default_stream_by_handle():
    """The NULL handle from inside another stream's context: outputs and kernel on the default stream."""
    fp8q = require_gpu()
    call = _calls(fp8q)["int8_quant_rows"]
    with torch.cuda.stream(torch.cuda.Stream()):
        q, s = call(0)
    torch.cuda.synchronize()
    assert _owner(q) == _owner(s) == torch.cuda.default_stream().cuda_stream == 0


@pytest.mark.parametrize("m", [3, 200])
def test_chain_on_a_stream_argument_alone(m):
    """The whole chain with stream=s from the default stream, whose own allocations and work go on meanwhile: the
    intermediate codes are dropped as soon as the next call is made."""
    fp8q = require_gpu()
    args = _chain_inputs(61, m)
    want = [t.clone() for t in _chain(fp8q, *args)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = _chain(fp8q, *args, stream=s)
        noise = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 18)]
        s.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
        assert all(bool((x == 0x55).all()) for x in noise)
