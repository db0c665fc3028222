"""The loss head among the operators of a step: its gradients through the sync, the norm and AdamW, and the example."""
import math
import os
import sys

import pytest
import torch

import gradient_sync_plan_gb300 as ddp
import loss_ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _inputs(tokens, vocab, dim, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(device="cuda", generator=gen)
    first = torch.randn(vocab, dim, **kw) * dim ** -0.5
    targets = [torch.randint(0, vocab, (n,), **kw) for n in tokens]
    for t in targets:
        t[::5] = -100
    return first, [torch.randn(n, dim, **kw).to(dtype) for n in tokens], targets


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,vocab,dim", [([40, 7, 1, 23], 90, 24), ([300, 513], 1001, 128)])
def test_a_step_from_the_loss_to_the_weights(tokens, vocab, dim, dtype):
    world = len(tokens)
    first, hidden, targets = _inputs(tokens, vocab, dim, dtype, 1)
    params = [[first.clone()] for _ in range(world)]
    weights = [first.to(dtype) for _ in range(world)]
    grads = [[torch.full_like(w, float("nan"))] for w in weights]
    state = [[[torch.zeros_like(first)] for _ in range(world)] for _ in range(2)]
    head = ddp.LossHead(weights, [g[0] for g in grads], max_tokens=max(tokens))
    code = ddp.BF16 if dtype == torch.bfloat16 else ddp.F32
    sync = ddp.SyncNormCall(grads, ddp.ddp_plan_buckets([first.numel()], code))
    update = ddp.AdamW(params, grads, *state, copies=[[w] for w in weights] if dtype == torch.bfloat16 else None)
    gh = [torch.empty_like(h) for h in hidden]
    for step in range(2):
        before = [w.clone() for w in weights]
        old = [params[r][0].double().clone() for r in range(world)]
        loss = head.cross_entropy_grad(hidden, targets, gh, reduction=ddp.DDP_LOSS_WORLD_MEAN)
        own = [g[0].clone() for g in grads]
        torch.cuda.synchronize()
        want = loss_ref.reference(hidden, before, targets, reduction="world_mean")
        loss_ref.check(want, loss, grad_hidden=gh, grad_weights=own)

        # the ranks' average is the gradient of the mean over all tokens: one rank that has them all
        joined = ddp.LossHead([before[0]], [torch.empty_like(before[0])], max_tokens=sum(tokens))
        total = joined.cross_entropy([torch.cat(hidden)], [torch.cat(targets)])
        norms = sync()
        torch.cuda.synchronize()
        mean = sum(w["grad_weights"] for w in want) / world
        # the ranks' bounds, and a rounding at each of world - 1 additions and the division, of sums below the magnitudes'
        bound = sum(w["weights_bound"] for w in want) / world
        bound += (world + 1) * loss_ref.half_step(dtype) * sum(w["grad_weights"].abs() + w["weights_bound"] for w in want) / world
        for r in range(world):
            assert bool(((grads[r][0].double() - mean).abs() <= bound).all())
            assert abs(float(norms[r]) / float(grads[r][0].double().norm()) - 1) < 1e-5
        every = loss_ref.reference([torch.cat(hidden)], [before[0]], [torch.cat(targets)])[0]
        assert abs(float(loss.double().mean()) - every["loss"]) <= max(w["loss_bound"] for w in want) + abs(every["loss"]) * 2.0 ** -22
        assert abs(float(total[0]) - every["loss"]) <= every["loss_bound"]

        if step == 0:
            update.step(1e-2, betas=(0.9, 0.95), norms=norms, max_norm=1.0)
            torch.cuda.synchronize()
            c = min(1.0, 1.0 / (float(norms[0]) + 1e-6))
            for r in range(world):
                # the first step: exp_avg / (1 - beta1) is the clipped gradient, and its square the other
                g = grads[r][0].double() * c
                after = old[r] - 1e-2 * g / (g.abs() + 1e-8)
                assert float((params[r][0].double() - after).abs().max()) < 1e-5
                if dtype == torch.bfloat16:
                    assert torch.equal(weights[r], params[r][0].bfloat16())          # the next step's weights
                else:
                    weights[r].copy_(params[r][0])


def test_micro_batches_accumulate_to_the_whole_batch():
    tokens, vocab, dim = [200], 300, 96
    first, hidden, targets = _inputs(tokens, vocab, dim, torch.float32, 2)
    grads = torch.zeros_like(first)
    head = ddp.LossHead([first], [grads], max_tokens=200)
    gh = [torch.empty(n, dim, device="cuda") for n in (120, 80)]
    parts = []
    for k, s in enumerate((slice(0, 120), slice(120, 200))):
        parts.append(head.cross_entropy_grad([hidden[0][s]], [targets[0][s].contiguous()], [gh[k]], reduction=ddp.DDP_LOSS_SUM,
                                             accumulate=True, out=torch.empty(1, device="cuda")))
    torch.cuda.synchronize()
    want = loss_ref.reference(hidden, [first], targets, reduction="sum")[0]
    assert abs(float(sum(parts)) - want["loss"]) <= want["loss_bound"] + abs(want["loss"]) * 2.0 ** -22
    off = (grads.double() - want["grad_weights"]).abs()
    assert bool((off <= 2 * want["weights_bound"]).all())             # a rounding more
    assert bool(((torch.cat(gh).double() - want["grad_hidden"]).abs() <= want["hidden_bound"]).all())


def test_two_heads_on_two_streams():
    runs = []
    for k in range(2):
        first, hidden, targets = _inputs([700], 2000, 192, torch.bfloat16, 3 + k)
        grads, gh = torch.empty_like(first.bfloat16()), torch.empty_like(hidden[0])
        runs.append((ddp.LossHead([first.bfloat16()], [grads], max_tokens=700), hidden, targets, grads, gh, torch.cuda.Stream()))
    alone = []
    for head, hidden, targets, grads, gh, _ in runs:
        head.cross_entropy_grad(hidden, targets, [gh])
        torch.cuda.synchronize()
        alone.append((grads.clone(), gh.clone(), head.loss.clone()))
    for _ in range(5):
        for head, hidden, targets, grads, gh, stream in runs:
            head.cross_entropy_grad(hidden, targets, [gh], stream=stream)
    torch.cuda.synchronize()
    for (head, _, _, grads, gh, _), want in zip(runs, alone):
        assert all(torch.equal(a, b) for a, b in zip((grads, gh, head.loss), want))
    assert ddp.ddp_device_status() == 0


def test_python_arguments():
    first, hidden, targets = _inputs([12, 5], 50, 16, torch.bfloat16, 5)
    weights = [first.bfloat16(), first.bfloat16()]
    head = ddp.LossHead(weights, [torch.empty_like(w) for w in weights], max_tokens=12, max_teacher=3)
    gh = [torch.empty_like(h) for h in hidden]
    good = dict(hidden=hidden, targets=targets)
    for bad in (dict(hidden=hidden[:1]), dict(hidden=[h.float() for h in hidden]), dict(hidden=[h.cpu() for h in hidden]),
                dict(hidden=[h[:, :8] for h in hidden]), dict(hidden=[hidden[0].t().contiguous().t(), hidden[1]]),
                dict(hidden=[hidden[0], torch.empty(5, 20, dtype=torch.bfloat16, device="cuda")[:, :16]]),
                dict(targets=targets[:1]), dict(targets=[t.int() for t in targets]), dict(targets=[t.cpu() for t in targets]),
                dict(targets=[targets[0], targets[0]]), dict(token_losses=[torch.empty(12, device="cuda")] * 3),
                dict(out=torch.empty(3, device="cuda")), dict(out=torch.empty(2))):
        with pytest.raises(ValueError):
            head.cross_entropy(**{**good, **bad})
    for bad in ([gh[0]], [gh[0], gh[0]], [g.float() for g in gh], [gh[0].t().contiguous().t(), gh[1]]):
        with pytest.raises(ValueError):
            head.cross_entropy_grad(hidden, targets, bad)
    logits, indices = [torch.zeros(n, 3, device="cuda") for n in (12, 5)], [torch.zeros(n, 3, dtype=torch.int64, device="cuda") for n in (12, 5)]
    for a, b in (([logits[0]], indices), (logits, [i.int() for i in indices]), (logits, [i[:, :2].contiguous() for i in indices]),
                 ([t.half() for t in logits], indices)):
        with pytest.raises((ValueError, TypeError)):
            head.distill(hidden, a, b)
    with pytest.raises(ddp.DDPError):
        head.distill(hidden, [torch.zeros(n, 4, device="cuda") for n in (12, 5)],
                     [torch.zeros(n, 4, dtype=torch.int64, device="cuda") for n in (12, 5)])        # more than max_teacher
    with pytest.raises(ddp.DDPError):
        ddp.LossHead(weights, max_tokens=4).cross_entropy(hidden, targets)                          # more than max_tokens
    torch.cuda.synchronize()
    assert ddp.ddp_device_status() == 0


@pytest.mark.parametrize("distill", [False, True])
def test_example(distill):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_tokens
    finally:
        sys.path.pop(0)
    losses, last = train_tokens.train(ranks=3, steps=4, distill=distill)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)
    extra = {}
    if distill:
        extra = dict(teacher=last["teacher"][0], indices=last["teacher"][1], temperature=2.0, alpha=0.5)
    want = loss_ref.reference(last["states"], last["weights"], last["targets"], reduction="world_mean", **extra)
    loss_ref.check(want, [x["loss"] for x in want], grad_hidden=last["grad_hidden"], grad_weights=last["head"])
