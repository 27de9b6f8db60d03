"""Adapters fine-tuned on a frozen 4-bit network, then several served at once.

    python examples/finetune_adapters.py [--steps 60] [--tokens 1024] [--features 1024]

A residual block y = x + fc2(silu(fc1(norm(x)))) has frozen NF4 layers; a
low-rank adapter beside each layer, and the norm, are trained with AdamW whose
states take 8 bits.  A second adapter is trained on other targets the same
way; then one batch in which each token names its adapter (or none) runs
through the block, as a server of many requests would run it.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_quantized_linear_i8lt_gb300 as I  # noqa: E402

DEV, DTYPE = "cuda", torch.bfloat16


class Block(torch.nn.Module):
    """x + fc2(silu(fc1(norm(x)))) with ``adapters`` adapters beside each layer."""

    def __init__(self, features: int, hidden: int, rank: int, adapters: int, seed: int = 0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def frozen(n, k):
            w = (torch.randn(n, k, generator=g) * k ** -0.5).to(DEV, DTYPE)
            return I.LinearNF4.from_float(w, double_quant=True)

        self.norm = I.LayerNorm(features, device=DEV)
        self.fc1 = I.LowRankAdapters(frozen(hidden, features), rank, adapters, device=DEV, dtype=DTYPE)
        self.fc2 = I.LowRankAdapters(frozen(features, hidden), rank, adapters, device=DEV, dtype=DTYPE)

    def forward(self, x, plan):
        return x + self.fc2(I.SiLUFunction.apply(self.fc1(self.norm(x), plan)), plan)


def train(block: Block, which: int, steps: int, tokens: int, features: int, lr: float = 3e-3):
    """Fits adapter ``which`` to targets of its own; returns the losses."""
    adapters = block.fc1.adapters
    index = torch.full((tokens,), which, dtype=torch.int32, device=DEV)
    plan = I.adapter_plan(index, adapters)                # one plan for all layers and steps of these tokens
    g = torch.Generator(device=DEV).manual_seed(100 + which)
    x = torch.randn(tokens, features, generator=g, device=DEV).to(DTYPE)
    shift = torch.randn(features, generator=g, device=DEV) * 0.5
    target = (x.float() + shift).to(DTYPE)
    opt = I.AdamW([p for p in block.parameters() if p.requires_grad], lr=lr, weight_decay=0.0, bits=8)
    losses = []
    for _ in range(steps):
        loss = ((block(x, plan) - target).float() ** 2).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]                     # read back once, at the end


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--features", type=int, default=1024)
    a = ap.parse_args(argv)
    block = Block(a.features, 2 * a.features + 64, rank=16, adapters=2)
    losses = []
    for which in (0, 1):
        losses.append(train(block, which, a.steps, a.tokens, a.features))
        print(f"adapter {which}: loss {losses[-1][0]:.4f} -> {losses[-1][-1]:.4f} in {a.steps} steps")
        block.norm.requires_grad_(False)                  # the norm is shared: trained with the first adapter only
    g = torch.Generator(device=DEV).manual_seed(7)
    x = torch.randn(a.tokens, a.features, generator=g, device=DEV).to(DTYPE)
    index = torch.randint(-1, 2, (a.tokens,), generator=g, device=DEV).int()
    with torch.no_grad():
        served = block(x, I.adapter_plan(index, 2))
        alone = [block(x, I.adapter_plan(torch.full_like(index, e), 2)) for e in (-1, 0, 1)]
    same = torch.stack(alone)[(index + 1).long(), torch.arange(a.tokens, device=DEV)]
    off = float((served.float() - same.float()).norm() / same.float().norm())
    print(f"a batch of {a.tokens} tokens with adapters -1, 0, 1 mixed: {off:.1e} from each adapter alone")
    return losses, off


if __name__ == "__main__":
    main()
