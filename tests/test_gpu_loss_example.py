"""The example's losses: what the loss head returned in its last step, against the definition on that step's inputs."""
import os
import sys

import pytest

import loss_ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("distill", [False, True])
def test_the_last_steps_losses(distill):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_tokens
    finally:
        sys.path.pop(0)
    losses, last = train_tokens.train(ranks=3, steps=3, distill=distill)
    extra = {}
    if distill:
        extra = dict(teacher=last["teacher"][0], indices=last["teacher"][1], temperature=2.0, alpha=0.5)
    want = loss_ref.reference(last["states"], last["weights"], last["targets"], reduction="world_mean", **extra)
    loss_ref.check(want, last["loss"], grad_hidden=last["grad_hidden"], grad_weights=last["head"])
    # what it reports is their mean over the ranks, rounded once more
    mean = sum(x["loss"] for x in want) / 3
    assert abs(losses[-1] - mean) <= max(x["loss_bound"] for x in want) + abs(mean) * 2.0 ** -22
