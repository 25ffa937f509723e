"""The gated feed-forward example: its gradients against 32-bit autograd, its training run and its 8-bit answers; and
the README's example of the operators."""

import importlib.util
import os
import re

import pytest
import torch

from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("gated_ffn_example", os.path.join(ROOT, "examples", "gated_ffn.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _rel(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def test_gradients_against_autograd():
    """An E4M3 code is off by at most 2^-4 of its value, 2.6% on average over a binade's steps; a result here has
    passed through at most six quantizations (x, the stacked weight, h, the down weight, dy, D), whose errors are
    independent: under 0.026 * sqrt(6) = 6.4%, held to 10%."""
    mod = _example()
    block = mod.GatedFFN(256, 384, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((256, 256), generator=gen, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn((256, 256), generator=gen, device="cuda", dtype=torch.bfloat16)
    y, saved = block.forward(x)
    dx, dw_gu, dw_d = block.backward(dy, saved)
    xr = x.float().requires_grad_()
    block.w_gu.requires_grad_()
    block.w_d.requires_grad_()
    ref = block.reference(xr)
    ref.backward(dy.float())
    assert _rel(y, ref.detach()) <= 0.1
    assert _rel(dx, xr.grad) <= 0.1 and _rel(dw_gu, block.w_gu.grad) <= 0.1 and _rel(dw_d, block.w_d.grad) <= 0.1


def _train_plain(mod, block, teacher, steps, tokens, lr, seed=0):
    """The example's training loop in plain FP32."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    params = [block.w_gu.clone().requires_grad_(), block.w_d.clone().requires_grad_()]
    momentum = [torch.zeros_like(p) for p in params]
    plain = mod.GatedFFN(*block.w_d.shape, seed=0)
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, block.w_d.shape[0]), generator=gen, device="cuda", dtype=torch.bfloat16)
        plain.w_gu, plain.w_d = params
        diff = plain.reference(x) - teacher.reference(x)
        losses.append(diff.square().mean().item())
        grads = torch.autograd.grad(diff.square().sum() / (2 * tokens), params)
        with torch.no_grad():
            for p, m, g in zip(params, momentum, grads):
                m.mul_(0.9).add_(g)
                p.sub_(m, alpha=lr)
    return losses


def test_training_follows_the_plain_run_and_served_answers():
    """Each step's gradient is off by some 6% in independent directions and the forward pass adds under 0.4% of the
    output's variance to the loss: the run follows the one in FP32, held to 10% of its loss.  8-bit rows are off by at
    most half a step of 1/127 of their largest value, about 3 standard deviations here: 0.7% of a value on average,
    four quantizations, held to 4%."""
    mod = _example()
    teacher, block, twin = mod.GatedFFN(256, 512, seed=1), mod.GatedFFN(256, 512, seed=2), mod.GatedFFN(256, 512, seed=2)
    losses = mod.train(block, teacher, steps=100, tokens=1024, lr=0.05)
    plain = _train_plain(mod, twin, teacher, steps=100, tokens=1024, lr=0.05)
    assert losses[-1] < losses[0] and abs(losses[-1] - plain[-1]) <= 0.1 * plain[-1], (losses[0], losses[-1], plain[-1])
    weights = block.for_serving()
    for n in (1, 5, 130):
        x = torch.randn((n, 256), device="cuda", dtype=torch.bfloat16)
        assert _rel(mod.serve(weights, x), block.reference(x)) <= 0.04


def test_served_answers_in_fp8():
    """Any number of tokens through the whole block: four quantizations (x, the stacked weight, h, the down weight) of
    2.6% each on average, independent: 5.2%, held to 8%.  The rows that pad h to whole tiles change nothing: in h's
    place the same rows with others behind them give the same answers."""
    mod = _example()
    fp8q = mod.fp8q
    block = mod.GatedFFN(256, 384, seed=5)
    weights = block.for_serving_fp8()
    for n in (1, 5, 128, 130, 300):
        x = torch.randn((n, 256), device="cuda", dtype=torch.bfloat16)
        y = mod.serve_fp8(weights, x)
        assert y.shape == (n, 256) and y.dtype == torch.bfloat16
        assert _rel(y, block.reference(x)) <= 0.08
        qx, sx = fp8q.fp8_quant_tile(x)
        full = torch.randn((n + -n % 128, 384), device="cuda", dtype=torch.bfloat16)
        full[:n] = fp8q.fp8_gemm_gated(qx, sx, *weights[:2])
        again = fp8q.fp8_gemm_blockscaled(fp8q.FPROP, *fp8q.fp8_quant_tile(full), *weights[2:])
        assert torch.equal(again[:n], y)


def test_readme_gated_example_runs():
    require_gpu()
    text = open(os.path.join(ROOT, "README.md")).read()
    block = re.search(r"## Gated feed-forward\n.*?```python\n(.*?)```", text, re.S).group(1)
    ns = {}
    exec(compile(block, "README.md (Gated feed-forward)", "exec"), ns)
    torch.cuda.synchronize()
    expect = {"h": ((8192, 18432), torch.bfloat16), "gu": ((8192, 36864), torch.bfloat16),
              "dw_gu": ((36864, 7168), torch.float32), "y1": ((1, 7168), torch.bfloat16)}
    for name, (shape, dtype) in expect.items():
        t = ns[name]
        assert tuple(t.shape) == shape and t.dtype == dtype, name
        assert bool(torch.isfinite(t.float()).all()), name
