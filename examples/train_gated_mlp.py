"""Trains a residual FP8 gated feed-forward block with the many-tensor AdamW
step and then serves it token by token.

    python examples/train_gated_mlp.py [--features 512] [--hidden 1408] [--bits 8]

The block learns a fixed random block of the same form, x + MLP(norm(x)), from
synthetic inputs. Per training step: forward and backward of the block under a
loss scale, the delayed-scaling update, one AdamW step over all parameters,
which also writes the E4M3 weight copies of the next forward pass.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_mixed_precision_reduce_gb300.adamw import AdamW  # noqa: E402
from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, features: int, hidden: int):
        super().__init__()
        self.norm = torch.nn.Parameter(torch.ones(features, device="cuda"))
        self.mlp = FP8GatedMLP(features, hidden)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        rms = torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)
        return x + self.mlp((x * rms * self.norm).to(torch.bfloat16)).to(x.dtype)


def run(features=512, hidden=1408, tokens=1000, steps=300, bits=8, lr=4e-3, log=print):
    """Returns the losses, and the largest difference between a token served
    alone and the same token in a batch, relative to the batch's output."""
    torch.manual_seed(0)
    teacher = [torch.randn(s, device="cuda") / s[1] ** 0.5 * 1.5
               for s in ((hidden, features), (hidden, features), (features, hidden))]
    block = Block(features, hidden)
    opt = AdamW(block.parameters(), lr=lr, weight_decay=0.01, max_norm=1.0, state_bits=bits, modules=[block.mlp])
    losses = []
    for step in range(steps):
        x = torch.randn((tokens, features), device="cuda")
        with torch.no_grad():
            n = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)
            target = x + (torch.nn.functional.silu(n @ teacher[0].T) * (n @ teacher[1].T)) @ teacher[2].T
        loss = (block(x) - target).pow(2).mean()
        opt.zero_grad()
        (loss * opt.loss_scale).sum().backward()
        block.mlp.update_scales()
        opt.step()
        losses.append(loss.detach())
        if step % 50 == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {loss.item():.4f}  gradient norm {(opt.grad_norm / opt.loss_scale).item():.4f}  "
                f"loss scale {opt.loss_scale.item():g}")
    with torch.no_grad():
        x = torch.randn((200, features), device="cuda")
        batch = block(x)
        alone = torch.cat([block(x[i:i + 1]) for i in range(8)])
        off = ((alone - batch[:8]).abs().max() / batch.abs().max()).item()
    log(f"8 tokens served one by one: within {off:.2g} of the batch's output")
    return torch.stack(losses).tolist(), off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--features", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1408)
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    args = ap.parse_args()
    run(args.features, args.hidden, args.tokens, args.steps, args.bits)
