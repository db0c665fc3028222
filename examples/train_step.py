"""One training step after another on N logical data-parallel ranks.

Each rank computes its own gradients of a small network on its own batch; the
sync averages them over the ranks and returns their global norm; the update
clips by that norm and writes the bf16 weights that the next forward uses.  The
step after the backward is two or three launches, and clipping takes no pass of its
own over the gradients.

    python examples/train_step.py [--ranks 4] [--steps 50]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gradient_sync_plan_gb300 as ddp

SHAPES = [(64, 256), (256,), (256, 256), (256,), (256, 8), (8,)]


def forward(weights, x):
    for i in range(0, len(weights), 2):
        x = x @ weights[i] + weights[i + 1]
        x = torch.relu(x) if i + 2 < len(weights) else x
    return x


def train(ranks: int = 4, steps: int = 50, max_norm: float = 1.0, seed: int = 0):
    """Returns the losses and the norms of every step, and the ranks' weights."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)
    target = rand(64, 8) * 0.2

    # every rank starts from the same weights: float32 masters, bf16 copies for the forward and backward
    start = [rand(*s) * (s[0] ** -0.5 if len(s) == 2 else 0.0) for s in SHAPES]
    params = [[w.clone() for w in start] for _ in range(ranks)]
    copies = [[w.bfloat16().requires_grad_() for w in row] for row in params]
    moments = [[[torch.zeros_like(w) for w in row] for row in params] for _ in range(2)]
    grads = [[torch.zeros_like(c) for c in row] for row in copies]

    numels = [w.numel() for w in start]
    sync = ddp.SyncNormCall(grads, ddp.ddp_plan_buckets(numels, ddp.BF16), algo=ddp.DDP_ALGO_VIEW)
    update = ddp.AdamW(params, grads, *moments, copies=[[c.detach() for c in row] for row in copies],
                       no_decay=[len(s) == 1 for s in SHAPES])

    losses, norms = [], []
    for _ in range(steps):
        loss = 0.0
        for r in range(ranks):
            x = rand(32, 64)
            out = forward(copies[r], x.bfloat16())
            err = (out.float() - x @ target).square().mean()
            for g, fresh in zip(grads[r], torch.autograd.grad(err, copies[r])):
                g.copy_(fresh)
            loss = loss + err.detach() / ranks
        norm = sync()                                      # averaged over the ranks, and their norm
        update.step(3e-3, betas=(0.9, 0.95), weight_decay=0.01, norms=norm, max_norm=max_norm)
        losses.append(loss)
        norms.append(norm[0].clone())
    return torch.stack(losses).tolist(), torch.stack(norms).tolist(), params


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    losses, norms, _ = train(a.ranks, a.steps)
    for k in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {k:4d}  loss {losses[k]:.4f}  gradient norm {norms[k]:.3f}")
    print(f"last       loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
