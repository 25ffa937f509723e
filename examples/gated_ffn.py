"""A gated feed-forward block, y = (silu(x Wg^T) * (x Wu^T)) Wd^T, trained in block-scaled FP8 and served in 8-bit
integers or in FP8:

    python examples/gated_ffn.py

A block with random weights learns to imitate another one.  Every product of the training step and every quantization
runs in the library's kernels; torch holds the master weights, the loss and the update.  The trained block then answers
single tokens and a batch with 8-bit weights and activations, integers or FP8.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_fp8_quant_amd as fp8q  # noqa: E402


class GatedFFN:
    """Master weights in FP32: gate and up stacked [2F][D], down [D][F]."""

    def __init__(self, d, f, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w_gu = torch.randn((2 * f, d), generator=gen, device="cuda") * d ** -0.5
        self.w_d = torch.randn((d, f), generator=gen, device="cuda") * f ** -0.5

    def reference(self, x):
        """The block in plain FP32."""
        f = self.w_d.shape[1]
        gu = x.float() @ self.w_gu.t()
        return (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]) @ self.w_d.t()

    def forward(self, x):
        """y (BF16) and what the backward pass needs: the codes of x, the weights and h that its products take, and
        the gate and up pre-activations.  x has a multiple of 128 rows, as Wgrad asks for."""
        qx, sx, qx_t, sx_t = fp8q.fp8_quant_tile_dual(x)
        qw, sw, qw_t, sw_t = fp8q.fp8_quant_block(self.w_gu, transposed=True)
        qd, sd, qd_t, sd_t = fp8q.fp8_quant_block(self.w_d, transposed=True)
        h, gu = fp8q.fp8_gemm_gated(qx, sx, qw, sw, save_gate_up=True)
        qh, sh, qh_t, sh_t = fp8q.fp8_quant_tile_dual(h)
        y = fp8q.fp8_gemm_blockscaled(fp8q.FPROP, qh, sh, qd, sd)
        return y, (qx_t, sx_t, qw_t, sw_t, qd_t, sd_t, qh_t, sh_t, gu)

    def backward(self, dy, saved):
        """Gradients of x (BF16), of the stacked gate and up weight and of the down weight (FP32)."""
        qx_t, sx_t, qw_t, sw_t, qd_t, sd_t, qh_t, sh_t, gu = saved
        qy, sy, qy_t, sy_t = fp8q.fp8_quant_tile_dual(dy)
        dh = fp8q.fp8_gemm_blockscaled(fp8q.DGRAD, qy, sy, qd_t, sd_t)
        dw_d = fp8q.fp8_gemm_blockscaled(fp8q.WGRAD, qy_t, sy_t, qh_t, sh_t, out_dtype=torch.float32)
        q, s, q_t, s_t = fp8q.fp8_gated_backward(dh, gu)
        dx = fp8q.fp8_gemm_blockscaled(fp8q.DGRAD, q, s, qw_t, sw_t)
        dw_gu = fp8q.fp8_gemm_blockscaled(fp8q.WGRAD, q_t, s_t, qx_t, sx_t, out_dtype=torch.float32)
        return dx, dw_gu, dw_d

    def for_serving(self):
        """8-bit codes of both weights with one scale for each output channel."""
        return (*fp8q.int8_quant_rows(self.w_gu), *fp8q.int8_quant_rows(self.w_d))

    def for_serving_fp8(self):
        """FP8 codes of both weights with one scale for each 128x128 block."""
        return (*fp8q.fp8_quant_block(self.w_gu), *fp8q.fp8_quant_block(self.w_d))


def serve(weights, x):
    """The block on any number of tokens, one included, in 8-bit integers."""
    qw, sw, qd, sd = weights
    qx, sx = fp8q.int8_quant_rows(x)
    qh, sh = fp8q.int8_quant_rows(fp8q.int8_gemm_gated(qx, sx, qw, sw))
    return fp8q.int8_gemm(qh, sh, qd, sd)


def serve_fp8(weights, x):
    """The block on any number of tokens, one included, in block-scaled FP8.  The down projection takes rows in whole
    tiles of 128: h is the head of a buffer of such tiles, whose other rows are zeros."""
    qw, sw, qd, sd = weights
    n = x.shape[0]
    qx, sx = fp8q.fp8_quant_tile(x)
    h = torch.zeros((n + -n % 128, qd.shape[1]), dtype=torch.bfloat16, device=x.device)
    fp8q.fp8_gemm_gated(qx, sx, qw, sw, h=h[:n])
    qh, sh = fp8q.fp8_quant_tile(h)
    return fp8q.fp8_gemm_blockscaled(fp8q.FPROP, qh, sh, qd, sd)[:n]


def train(block, teacher, steps, tokens, lr=0.02, seed=0, log=None):
    """Plain momentum descent on the mean squared error; returns the loss of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    d = block.w_d.shape[0]
    momentum = [torch.zeros_like(block.w_gu), torch.zeros_like(block.w_d)]
    losses = []
    for step in range(steps):
        x = torch.randn((tokens, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        target = teacher.reference(x)
        y, saved = block.forward(x)
        diff = y.float() - target
        losses.append(diff.square().mean().item())
        _, *grads = block.backward((diff * (1.0 / tokens)).to(torch.bfloat16), saved)
        for w, m, g in zip((block.w_gu, block.w_d), momentum, grads):
            m.mul_(0.9).add_(g)
            w.sub_(m, alpha=lr)
        if log and step % 50 == 0:
            log(f"step {step:4d}  loss {losses[-1]:.5f}")
    return losses


def main():
    d, f, tokens = 512, 1024, 2048
    teacher, block = GatedFFN(d, f, seed=1), GatedFFN(d, f, seed=2)
    losses = train(block, teacher, steps=400, tokens=tokens, lr=0.1, log=print)
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}")
    for form, answer, weights in (("8-bit integers", serve, block.for_serving()), ("FP8", serve_fp8, block.for_serving_fp8())):
        for n in (1, 17, 300):
            x = torch.randn((n, d), device="cuda", dtype=torch.bfloat16)
            y, ref = answer(weights, x).float(), block.reference(x)
            print(f"served {n:3d} tokens in {form}: relative error {(y - ref).norm() / ref.norm():.4f}")


if __name__ == "__main__":
    main()
