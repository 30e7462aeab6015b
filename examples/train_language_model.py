"""Trains a small language model of FP8 blocks and then continues texts with it.

    python examples/train_language_model.py [--features 256] [--hidden 704] [--blocks 2] [--steps 200]

Embedding from an E4M3 table, residual blocks whose norm, residual addition and cast are
one kernel, a head that gives log probabilities and takes their gradient as E5M2 codes,
AdamW over all of it. The texts are synthetic: each token is one of a few that follow the
one before it. Without attention the model sees one token at a time, which is all that
they ask for.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_mixed_precision_reduce_gb300.adamw import AdamW  # noqa: E402
from fp8_mixed_precision_reduce_gb300.embedding import TokenEmbedding  # noqa: E402
from fp8_mixed_precision_reduce_gb300.gated_mlp import FP8GatedMLP  # noqa: E402
from fp8_mixed_precision_reduce_gb300.lm_head import FP8LMHead  # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, vocab: int, features: int, hidden: int, blocks: int):
        super().__init__()
        self.embedding = TokenEmbedding(vocab, features, scale=features ** 0.5, fp8=True)
        self.blocks = torch.nn.ModuleList(FP8GatedMLP(features, hidden, norm_eps=1e-6) for _ in range(blocks))
        self.head = FP8LMHead(features, vocab, norm_eps=1e-6)

    def fp8_modules(self):
        return [self.embedding, *self.blocks, self.head]

    def stream(self, ids):
        x, residual = self.embedding(ids), None
        for block in self.blocks:
            x, residual = block(x, residual)
        return x, residual

    def forward(self, ids, targets, entropy: bool = False):
        x, residual = self.stream(ids)
        return self.head(x, targets, residual, entropy)

    def top(self, ids, k: int = 1):
        x, residual = self.stream(ids)
        return self.head.top(x, k, residual)


def texts(follow, batch, length):
    """Token t is followed by one of follow[t]."""
    ids = [torch.randint(0, follow.shape[0], (batch,), device="cuda")]
    for _ in range(length):
        pick = torch.randint(0, follow.shape[1], (batch,), device="cuda")
        ids.append(follow[ids[-1], pick])
    return torch.stack(ids, 1)


def run(vocab=1000, features=256, hidden=704, blocks=2, batch=32, length=63, steps=200, lr=3e-3, bits=8, log=print):
    """Returns the losses, and the share of greedy next tokens that the texts allow."""
    torch.manual_seed(0)
    follow = torch.randint(0, vocab, (vocab, 3), device="cuda")
    model = Model(vocab, features, hidden, blocks)
    opt = AdamW(model.parameters(), lr=lr, weight_decay=0.01, max_norm=1.0, state_bits=bits, modules=model.fp8_modules())
    losses = []
    for step in range(steps):
        ids = texts(follow, batch, length)
        logprob = model(ids[:, :-1], ids[:, 1:])
        loss = -logprob.mean()
        opt.zero_grad()
        (loss * opt.loss_scale).sum().backward()
        for module in model.fp8_modules():
            module.update_scales()
        opt.step()
        losses.append(loss.detach())
        if step % 50 == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {loss.item():.4f}  loss scale {opt.loss_scale.item():g}")
    with torch.no_grad():
        ids = torch.randint(0, vocab, (64,), device="cuda")
        _, tokens = model.top(ids, 1)
        good = (follow[ids] == tokens).any(1).float().mean().item()
    log(f"{good:.0%} of the next tokens are among those that may follow (the entropy of a text is {torch.tensor(3.0).log():.4f})")
    return torch.stack(losses).tolist(), good


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--features", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=704)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    args = ap.parse_args()
    run(args.vocab, args.features, args.hidden, args.blocks, steps=args.steps, bits=args.bits)
