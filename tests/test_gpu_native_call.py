"""The native call path takes the usual calls of the gated feed-forward operators, answers what the ctypes path does, and
lets other threads run meanwhile."""

import sys
import threading
import time

import pytest
import torch

from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

F32, BF, I8 = torch.float32, torch.bfloat16, torch.int8


def _ints(rows, cols):
    buf = torch.randint(-128, 128, (rows, -(-cols // 16) * 16), device="cuda", dtype=I8)
    return buf[:, :cols], torch.rand(rows, device="cuda") * 1e-2


def _codes(fp8q, m, f, k):
    x, w = torch.randn(m, k, device="cuda"), torch.randn(2 * f, k, device="cuda") * 0.05
    return (*fp8q.fp8_quant_tile(x), *fp8q.fp8_quant_block(w))


def _calls(fp8q):
    """(entry point, arguments, keywords, the arguments of its native form)."""
    calls = []
    for m, n, k in [(1, 32, 48), (1, 37, 1001), (5, 40, 333), (130, 200, 256)]:
        (a, sa), (b, sb), bias = _ints(m, k), _ints(2 * n, k), torch.randn(2 * n, device="cuda")
        calls += [("int8_gemm", (a, sa, b, sb), dict(bias=bias, out_dtype=F32), (a, sa, b, sb, bias, fp8q.F32)),
                  ("int8_gemm", (a, sa, b, sb), {}, (a, sa, b, sb, None, fp8q.BF16)),
                  ("int8_gemm_gated", (a, sa, b, sb), dict(act=fp8q.ACT_GELU_TANH), (a, sa, b, sb, 1, fp8q.BF16))]
    for rows, cols in [(1, 37), (3, 1001), (17, 64)]:
        for dtype in (BF, F32):
            x = torch.randn(rows, -(-cols // 8) * 8, device="cuda").to(dtype)[:, :cols]
            calls.append(("int8_quant_rows", (x,), {}, (x,)))
    for m, f, k in [(1, 128, 256), (133, 256, 384)]:
        ops = _codes(fp8q, m, f, k)
        calls += [("fp8_gemm_gated", ops, {}, (*ops, 0, fp8q.BF16, False)),
                  ("fp8_gemm_gated", (ops[0].view(torch.float8_e4m3fn), *ops[1:]), dict(out_dtype=F32, save_gate_up=True),
                   (ops[0].view(torch.float8_e4m3fn), *ops[1:], 0, fp8q.F32, True))]
        for dtype in (BF, F32):
            dh, gu = torch.randn(m, f, device="cuda").to(dtype), torch.randn(m, 2 * f, device="cuda").to(dtype)
            calls.append(("fp8_gated_backward", (dh, gu), dict(act=1, mode=fp8q.POW2), (dh, gu, 1, fp8q.POW2)))
    return calls


def _list(r):
    return [r] if torch.is_tensor(r) else list(r)


def test_native_call_takes_the_usual_calls_and_answers_like_ctypes(monkeypatch):
    fp8q = require_gpu()
    from precision_fp8_quant_amd import ffn
    native = ffn._native
    assert native is not None, "_ffn_call.so is not built or was refused"
    calls = _calls(fp8q)
    assert {c[0] for c in calls} == set(ffn.SIGNATURES)
    for name, args, kw, native_args in calls:
        got = getattr(native, name)(*native_args)
        assert got is not None and not isinstance(got, int), (name, [getattr(a, "shape", a) for a in args], got)
        public = getattr(fp8q, name)(*args, **kw)
        monkeypatch.setattr(ffn, "_native", None)
        want = getattr(fp8q, name)(*args, **kw)
        monkeypatch.setattr(ffn, "_native", native)
        assert len(_list(got)) == len(_list(want))
        for x, y, z in zip(_list(got), _list(want), _list(public)):
            assert x.shape == y.shape == z.shape and x.stride() == y.stride() == z.stride() and x.dtype == y.dtype, name
            assert torch.equal(x, y) and torch.equal(z, y), name


def test_native_call_lets_other_threads_run():
    """The allocator and the launch run without the interpreter's lock, as in a ctypes call: a thread that waits for the
    lock gets it from a loop of native calls, which with this switch interval gives it up nowhere else."""
    fp8q = require_gpu()
    from precision_fp8_quant_amd import ffn
    (a, sa), (b, sb) = _ints(1, 64), _ints(64, 64)
    args = (a, sa, b, sb, None, fp8q.BF16)
    ffn._native.int8_gemm(*args)
    torch.cuda.synchronize()
    ran, gate = [], threading.Lock()
    gate.acquire()

    def other():
        gate.acquire()                                       # then it needs nothing but the interpreter's lock
        ran.append(True)
    t = threading.Thread(target=other)
    before = sys.getswitchinterval()
    try:
        sys.setswitchinterval(1000.0)
        t.start()
        time.sleep(0.1)                                      # the thread is at its gate
        gate.release()
        calls, kept = 0, []
        while not ran and calls < 20000:
            kept.append(ffn._native.int8_gemm(*args))         # freeing a tensor gives the lock up, too
            calls += 1
        assert ran, "no other thread ran during 20000 native calls"
    finally:
        sys.setswitchinterval(before)
        t.join()
    torch.cuda.synchronize()
