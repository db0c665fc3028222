"""A small language model on N logical data-parallel ranks, from its loss to its weights.

Each rank reads its own tokens, as many as it happens to have.  The loss head computes cross entropy over the vocabulary
from the hidden states and the tied embedding's weights, never keeping logits, and writes the gradients of the hidden
states, which torch's backward takes from there, and of the head, to which the embedding's own gradient is added.  The
sync averages the ranks' gradients (losses weighted so that this is the mean over all tokens) and returns their norm;
the update clips by it and writes the bf16 weights of the next step.  With --distill a student learns from a frozen
teacher's top logits instead.

    python examples/train_tokens.py [--ranks 4] [--steps 50] [--distill]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gradient_sync_plan_gb300 as ddp

VOCAB, DIM, TOP = 211, 64, 8
SHAPES = [(VOCAB, DIM), (DIM, DIM), (DIM, DIM)]


def hidden_states(weights, tokens):
    x = weights[0][tokens]
    return x + torch.relu(x @ weights[1]) @ weights[2]


def train(ranks: int = 4, steps: int = 50, distill: bool = False, max_norm: float = 1.0, seed: int = 0):
    """Returns every step's mean loss over all tokens, and the last step's inputs, losses and gradients of every rank."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)
    follows = torch.randperm(VOCAB, device="cuda", generator=gen)         # the language: each token has a successor

    start = [rand(*s) * s[1] ** -0.5 for s in SHAPES]
    params = [[w.clone() for w in start] for _ in range(ranks)]
    copies = [[w.bfloat16().requires_grad_() for w in row] for row in params]
    moments = [[[torch.zeros_like(w) for w in row] for row in params] for _ in range(2)]
    grads = [[torch.zeros_like(c) for c in row] for row in copies]

    most = 64
    head = ddp.LossHead([row[0].detach() for row in copies], [row[0] for row in grads], max_tokens=most, max_teacher=TOP)
    sync = ddp.SyncNormCall(grads, ddp.ddp_plan_buckets([w.numel() for w in start], ddp.BF16), algo=ddp.DDP_ALGO_VIEW)
    update = ddp.AdamW(params, grads, *moments, copies=[[c.detach() for c in row] for row in copies])

    losses, last = [], None
    for _ in range(steps):
        inputs = [torch.randint(0, VOCAB, (most - 9 * r,), device="cuda", generator=gen) for r in range(ranks)]
        targets = [follows[t] for t in inputs]
        for t in targets:
            t[::7] = -100                                                 # tokens that are not learned, as a prompt's
        hidden = [hidden_states(copies[r], inputs[r]) for r in range(ranks)]
        states = [h.detach() for h in hidden]
        grad_hidden = [torch.empty_like(s) for s in states]
        how = dict(targets=targets, reduction=ddp.DDP_LOSS_WORLD_MEAN)
        teacher = None
        if distill:
            # a teacher that knows the language: the successor first, then some others
            indices = [(follows[t].unsqueeze(1) + torch.arange(TOP, device="cuda")) % VOCAB for t in inputs]
            logits = [torch.linspace(6.0, -6.0, TOP, device="cuda").expand(t.numel(), TOP).contiguous() for t in inputs]
            teacher = (logits, indices)
            loss = head.distill_grad(states, logits, indices, grad_hidden, temperature=2.0, alpha=0.5, **how)
        else:
            loss = head.cross_entropy_grad(states, grad_hidden=grad_hidden, **how)
        if last is None or len(losses) == steps - 1:
            last = dict(states=states, targets=targets, teacher=teacher, weights=[row[0].detach().clone() for row in copies],
                        head=[row[0].clone() for row in grads], grad_hidden=grad_hidden, loss=loss.clone())
        for r in range(ranks):
            fresh = torch.autograd.grad(hidden[r], copies[r], grad_hidden[r])
            grads[r][0] += fresh[0]                                       # the embedding's rows, beside the head's
            for g, f in zip(grads[r][1:], fresh[1:]):
                g.copy_(f)
        norms = sync()
        update.step(1e-2, betas=(0.9, 0.95), weight_decay=0.01, norms=norms, max_norm=max_norm)
        losses.append(loss.mean())
    return torch.stack(losses).tolist(), last


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--distill", action="store_true")
    a = ap.parse_args()
    losses, _ = train(a.ranks, a.steps, a.distill)
    for k in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {k:4d}  loss {losses[k]:.4f}")
    print(f"last       loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
