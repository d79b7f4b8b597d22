"""A small patch transformer trained as a denoiser with the SSIM loss: the loss,
the residual norms and the gradient clipping in one training step.

    python examples/train_denoiser.py [--steps 200] [--batch 8] [--dim 256] [--depth 4]

Clean images are the smooth synthetic renders of workloads.splat_render (64 x 64),
the input is a copy with Gaussian noise of a random strength.  Tokens are 8 x 8
patches; a block mixes tokens, then channels; its norms and gates are
conditioned on the noise strength.  The residual stream is float32, what lies
between the norms bfloat16.  Matrix products are torch's; everything between
them, the loss and the clipping are this package's kernels.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402
import torch.nn.functional as F  # noqa: E402

from differentiable_image_quality_gb300 import (  # noqa: E402
    clip_grad_norm_, fused_residual_norm, fused_ssim)
from workloads import splat_render  # noqa: E402

SIZE, PATCH = 64, 8
TOKENS, PATCH_DIM = (SIZE // PATCH) ** 2, 3 * PATCH * PATCH


def linear(x, layer):
    return F.linear(x, layer.weight.to(x.dtype), layer.bias.to(x.dtype))


class Denoiser(torch.nn.Module):
    def __init__(self, dim: int, depth: int):
        super().__init__()
        self.dim, self.depth = dim, depth
        self.embed = torch.nn.Linear(PATCH_DIM, dim)
        self.position = torch.nn.Parameter(0.02 * torch.randn(TOKENS, dim))
        # per sub-block from the noise strength: gate, and scale and shift of the norm before
        self.condition = torch.nn.Linear(16, (2 * depth * 3 + 2) * dim)
        torch.nn.init.normal_(self.condition.weight, std=0.02)
        self.tokens = torch.nn.ModuleList(
            torch.nn.Linear(TOKENS, TOKENS) for _ in range(depth))
        self.up = torch.nn.ModuleList(torch.nn.Linear(dim, 2 * dim) for _ in range(depth))
        self.down = torch.nn.ModuleList(torch.nn.Linear(2 * dim, dim) for _ in range(depth))
        self.post = torch.nn.ParameterList(  # as differences from one, like the norms before
            torch.nn.Parameter(torch.zeros(dim)) for _ in range(2 * depth))
        self.head = torch.nn.Linear(dim, PATCH_DIM)
        torch.nn.init.zeros_(self.head.weight)
        torch.nn.init.zeros_(self.head.bias)

    def forward(self, noisy: torch.Tensor, strength: torch.Tensor) -> torch.Tensor:
        n = noisy.shape[0]
        patches = F.unfold(noisy, PATCH, stride=PATCH).transpose(1, 2)
        x = self.embed(patches) + self.position
        waves = strength[:, None] * torch.arange(1, 9, device=x.device) * 6.0
        mod = self.condition(torch.cat([waves.sin(), waves.cos()], 1))
        mod = iter(mod.chunk(2 * self.depth * 3 + 2, dim=1))  # [samples, dim], a stride apart
        norm = dict(pre_norm="layer", weight_offset=1.0)
        scale, shift = next(mod), next(mod)
        # the norm before the first block; after that each block's own call ends it
        # and begins the next
        x, u = fused_residual_norm(x, pre_weight=scale, pre_bias=shift, u_dtype=torch.bfloat16,
                                   **norm)
        for i in range(2 * self.depth):
            if i % 2 == 0:
                y = linear(u.transpose(1, 2), self.tokens[i // 2]).transpose(1, 2).contiguous()
            else:
                y = linear(F.gelu(linear(u, self.up[i // 2])), self.down[i // 2])
            gate, scale, shift = next(mod), next(mod), next(mod)
            x, u = fused_residual_norm(x, y, gate, post_norm="rms", post_weight=self.post[i],
                                       pre_weight=scale, pre_bias=shift, residual_scale=1.0, **norm)
        out = F.fold(linear(u, self.head).float().transpose(1, 2), SIZE, PATCH, stride=PATCH)
        return noisy + strength[:, None, None, None] * out  # out: minus the noise, in its own units


def batches(batch: int, seed: int = 0):
    """Clean and noisy images, and the strength of the noise, on the GPU."""
    rng = np.random.default_rng(seed)
    pool = torch.from_numpy(splat_render(rng, 32, 3, SIZE, SIZE, blobs=40, s_lo=3.0,
                                         s_hi=15.0).astype(np.float32)).cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    while True:
        pick = torch.randint(0, pool.shape[0], (batch,), generator=gen, device="cuda")
        clean = pool[pick]
        strength = 0.05 + 0.1 * torch.rand(batch, generator=gen, device="cuda")
        noise = torch.randn(clean.shape, generator=gen, device="cuda")
        yield clean, clean + strength[:, None, None, None] * noise, strength


def train(steps: int = 200, batch: int = 8, dim: int = 256, depth: int = 4, lr: float = 1e-3,
          max_norm: float = 1.0, report=print) -> list:
    """Trains and returns the loss of every step."""
    torch.manual_seed(0)
    model = Denoiser(dim, depth).cuda()
    optimizer = torch.optim.AdamW(model.parameters(), lr=lr)
    data, losses = batches(batch), []
    for step in range(steps):
        clean, noisy, strength = next(data)
        restored = model(noisy, strength)
        loss = 1 - fused_ssim(restored.contiguous(), clean, padding="valid")
        optimizer.zero_grad(set_to_none=True)
        loss.backward()
        norm = clip_grad_norm_(model.parameters(), max_norm)
        optimizer.step()
        losses.append(loss.detach())
        if step % 20 == 0 or step == steps - 1:
            report(f"step {step:4d}  1 - SSIM {losses[-1].item():.4f}  "
                   f"gradient norm {norm.item():.4f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--depth", type=int, default=4)
    a = ap.parse_args()
    train(a.steps, a.batch, a.dim, a.depth)
