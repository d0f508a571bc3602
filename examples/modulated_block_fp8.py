"""A modulated MLP block of a transformer on frozen E4M3 weights with a scale for each 128 x 128 block, trained through:

    n = layer_norm(x) * (1 + scale) + shift     scale and shift of each image; straight into E4M3 codes
    y = x + fc2(gelu(fc1(n)))                   two block-scaled layers

and backwards, for what produces scale and shift (a conditioning network, an adapter) and what lies before the block:

    dh = dy fc2^T,  da = dh gelu'(a),  dn = da fc1^T        the same layers on transposed weights
    dx = dy + .., dscale, dshift                            the norm's gradient, from the forward's mean and rstd

Codes count as the values they stand for.  Prints the error of y and of each gradient against fp32 and the time of a pass.

    python examples/modulated_block_fp8.py [--images 2] [--rows 512] [--channels 768]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_diffusion_model_amd import svdq  # noqa: E402
from bit_diffusion_model_amd.workloads import bf16_bits_from_f64, bf16_bits_to_f32  # noqa: E402


class Mlp(torch.autograd.Function):
    """fc2(gelu(fc1(layer_norm(x) (1 + scale) + shift))) on x [B][S][C] bf16, scale and shift [B][C]."""

    @staticmethod
    def forward(ctx, x, scale, shift, layers):
        fc1, fc2 = layers[:2]
        norm = svdq.LayerNorm(x.shape[-1], scale.detach(), shift.detach(), 1e-6, one_plus=True)
        stats = norm.alloc_stats(x)
        a = norm.forward_linear(x, fc1, svdq.BF16, stats=stats)
        y = fc2.forward(torch.nn.functional.gelu(a), svdq.BF16).view(x.shape)
        ctx.save_for_backward(x, scale, shift, a, *stats)
        ctx.norm, ctx.layers = norm, layers
        return y

    @staticmethod
    def backward(ctx, dy):
        x, _, _, a, mean, rstd = ctx.saved_tensors
        fc1_t, fc2_t = ctx.layers[2:]
        dh = fc2_t.forward(dy.reshape(-1, dy.shape[-1]), svdq.F32)
        da = torch.ops.aten.gelu_backward(dh, a.float())
        dn = fc1_t.forward(da, svdq.BF16).view(x.shape)
        dx, dscale, dshift = ctx.norm.backward(dn, x, (mean, rstd))
        return dx, dscale, dshift, None


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--images", type=int, default=2)
    ap.add_argument("--rows", type=int, default=512)
    ap.add_argument("--channels", type=int, default=768)
    args = ap.parse_args()
    rng, B, S, C = np.random.default_rng(0), args.images, args.rows, args.channels
    torch.manual_seed(0)

    def packed(K, N):
        bits = bf16_bits_from_f64(rng.standard_normal((K, N)) / np.sqrt(K))
        bias = (0.1 * rng.standard_normal(N)).astype(np.float32)
        lin = svdq.Fp8Linear.from_weights(bits, bias)
        return lin, torch.from_numpy(bf16_bits_to_f32(bits)).cuda(), lin.bias

    (fc1, w1, b1), (fc2, w2, b2) = packed(C, 4 * C), packed(4 * C, C)
    layers = (fc1, fc2, fc1.transposed(), fc2.transposed())
    x = (3 * torch.randn(B, S, C, device="cuda") + 1).bfloat16().requires_grad_()
    scale, shift = ((0.3 * torch.randn(B, C, device="cuda")).requires_grad_() for _ in range(2))
    dy = torch.randn(B, S, C, device="cuda").bfloat16()

    def step():
        y = x + Mlp.apply(x, scale, shift, layers)
        return (y, *torch.autograd.grad(y, (x, scale, shift), dy))

    xr, sr, tr = (t.detach().float().requires_grad_() for t in (x, scale, shift))
    n = torch.nn.functional.layer_norm(xr, (C,), eps=1e-6) * (1 + sr[:, None]) + tr[:, None]
    mlp = torch.nn.functional.gelu(n.view(-1, C) @ w1 + b1) @ w2 + b2
    want = (mlp.detach().view(B, S, C), *torch.autograd.grad(mlp, (xr, sr, tr), dy.float().view(-1, C)))
    y, dx, dscale, dshift = step()
    got = (y - x, dx - dy, dscale, dshift)  # the MLP's part
    errors = {k: float((g.detach().float() - w).norm() / w.norm()) for k, g, w in zip(("y", "dx", "dscale", "dshift"), got, want)}
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(5):
        step()
    start.record()
    for _ in range(20):
        step()
    end.record()
    end.synchronize()
    print(", ".join(f"{k}: relative error {v:.2e}" for k, v in errors.items()))
    print(f"{B} images of {S} rows, {C} channels: {start.elapsed_time(end) / 20 * 1e3:.0f} us forward and backward")
    return errors


if __name__ == "__main__":
    main()
