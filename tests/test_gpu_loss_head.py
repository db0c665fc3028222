"""The loss head on the GPU against its definition in float64: cross entropy and distillation, losses and gradients."""
import pytest
import torch

import gradient_sync_plan_gb300 as ddp
import loss_ref
from loss_ref import IGNORE, LOSS

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _inputs(tokens, vocab, dim, dtype=BF16, ignored=0.0, seed=0, teacher=0, lean=6.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(device="cuda", generator=gen)
    x = dict(weights=[], hidden=[], targets=[], teacher=[], indices=[])
    for n in tokens:
        w = (torch.randn(vocab, dim, **kw) * dim ** -0.5).to(dtype)
        y = torch.randint(0, vocab, (n,), **kw)
        x["weights"].append(w)
        x["hidden"].append((torch.randn(n, dim, **kw) + torch.rand(n, 1, **kw) * lean * w[y].float()).to(dtype))
        x["targets"].append(y.masked_fill(torch.rand(n, **kw) < ignored, IGNORE))
        if teacher:
            order = torch.rand(n, vocab, **kw).argsort(1)[:, :teacher]
            x["indices"].append(order.contiguous())
            x["teacher"].append(torch.randn(n, teacher, **kw) * 3)
    return x


class Run:
    """A head over the inputs, with outputs that hold NaN before a call."""

    def __init__(self, x, grads=True, max_tokens=None, max_teacher=None):
        self.x = x
        self.tokens = [h.shape[0] for h in x["hidden"]]
        self.gw = [torch.full_like(w, float("nan")) for w in x["weights"]] if grads else None
        k = x["teacher"][0].shape[1] if x["teacher"] else 0
        self.head = ddp.LossHead(x["weights"], self.gw, max_tokens=max_tokens or max(self.tokens + [1]),
                                 max_teacher=k if max_teacher is None else max_teacher)
        self.head._workspace.fill_(255)                  # a program's memory holds anything: NaN here
        self.losses = [torch.full((n,), float("nan"), device="cuda") for n in self.tokens]
        self.gh = [torch.full((n, w.shape[1]), float("nan"), dtype=w.dtype, device="cuda")
                   for n, w in zip(self.tokens, x["weights"])]

    def ce(self, grad=True, reduction="mean", **kw):
        args = dict(reduction=LOSS[reduction], token_losses=self.losses, **kw)
        if grad:
            return self.head.cross_entropy_grad(self.x["hidden"], self.x["targets"], self.gh, **args)
        return self.head.cross_entropy(self.x["hidden"], self.x["targets"], **args)

    def distill(self, grad=True, targets=True, reduction="mean", **kw):
        args = dict(reduction=LOSS[reduction], token_losses=self.losses, targets=self.x["targets"] if targets else None, **kw)
        if grad:
            return self.head.distill_grad(self.x["hidden"], self.x["teacher"], self.x["indices"], self.gh, **args)
        return self.head.distill(self.x["hidden"], self.x["teacher"], self.x["indices"], **args)

    def check(self, loss, grad=True, targets=True, distill=False, **kw):
        torch.cuda.synchronize()
        assert ddp.ddp_device_status() == 0
        extra = dict(teacher=self.x["teacher"], indices=self.x["indices"]) if distill else {}
        want = loss_ref.reference(self.x["hidden"], self.x["weights"], self.x["targets"] if targets else None, **extra, **kw)
        loss_ref.check(want, loss, self.losses, self.gh if grad else None, self.gw if grad else None)
        return want


SIZES = [([1], 100, 32), ([1], 1, 8), ([3], 2, 1), ([16, 7], 100, 32), ([128], 256, 64), ([129], 257, 65), ([130, 1, 64], 513, 96),
         ([300], 1000, 256), ([257, 300], 391, 515), ([40], 5003, 7), ([33], 127, 1000)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,vocab,dim", SIZES)
def test_cross_entropy_losses(tokens, vocab, dim, dtype):
    run = Run(_inputs(tokens, vocab, dim, dtype, ignored=0.2, seed=len(tokens) + vocab), grads=False)
    run.check(run.ce(grad=False, reduction="sum"), grad=False, reduction="sum")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,vocab,dim", SIZES)
def test_cross_entropy_gradients(tokens, vocab, dim, dtype):
    run = Run(_inputs(tokens, vocab, dim, dtype, ignored=0.2, seed=vocab + dim))
    run.check(run.ce(reduction="world_mean", scale=3.0), reduction="world_mean", scale=3.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("temperature,alpha,targets", [(1.0, 1.0, False), (2.0, 1.0, False), (1.0, 0.3, True), (2.5, 0.7, True),
                                                       (0.5, 1.0, True)])
@pytest.mark.parametrize("tokens,vocab,dim,k", [([5], 40, 32, 1), ([16, 7], 100, 32, 8), ([130, 200], 777, 128, 64),
                                                ([64], 300, 66, 256)])
def test_distillation(tokens, vocab, dim, k, temperature, alpha, targets, dtype):
    x = _inputs(tokens, vocab, dim, dtype, ignored=0.2 if targets else 0.0, seed=k + dim, teacher=k)
    how = dict(temperature=temperature, alpha=alpha, targets=targets)
    run = Run(x)
    run.check(run.distill(reduction="mean", **how), distill=True, reduction="mean", **how)
    alone = Run(x, grads=False)
    alone.check(alone.distill(grad=False, reduction="world_mean", **how), grad=False, distill=True, reduction="world_mean", **how)
