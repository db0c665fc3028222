"""Gradients of the loss head where the vocabulary goes in pieces, the depth in parts, or a call has no tokens.

Bounds are those of loss_ref.py, computed for a thousand tokens at a time; where exponentials are kept in 16 bits they are
off by 2^-11 of them more, which counts r times for a softmax whose exponentials are the other's to the power r.
"""
import pytest
import torch

import gradient_sync_plan_gb300 as ddp
import loss_ref
from loss_ref import IGNORE, half_step, sum_steps

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF16, F32])


def _check_rank(x, r, out, f, scale, alpha, tau, old):
    """Rank r's losses and gradients against float64, in runs of 1024 learned tokens; f: the reduction's factor.  Returns the
    float64 loss."""
    dtype = x["weights"][r].dtype
    hard, soft = alpha < 1.0, alpha > 0.0
    keep = (x["targets"][r] != IGNORE).nonzero()[:, 0]
    w = x["weights"][r].double()
    vocab, dim = w.shape
    gw, ew = torch.zeros_like(w), torch.zeros_like(w)
    s, total = scale * f, 0.0
    bits = 2.0 ** -8 if dtype == BF16 else 2.0 ** -22            # of a logit's gradient, for the products
    for a in range(0, len(keep), 1024):
        k = keep[a:a + 1024]
        h, y = x["hidden"][r][k].double(), x["targets"][r][k].unsqueeze(1)
        z = h @ w.t()
        e_logit = float((h.abs() @ w.abs().t()).max()) * sum_steps(dtype, dim)
        e = (2 * e_logit + (float(z.abs().max()) + 40) * 2.0 ** -21) * max(1.0, 1 / tau)
        loss, e_loss = torch.zeros(len(k), dtype=torch.float64, device="cuda"), 0.0
        dz, mass = torch.zeros_like(z), torch.zeros_like(z)
        if hard:
            logp = torch.log_softmax(z, 1)
            loss -= (1 - alpha) * logp.gather(1, y).squeeze(1)
            p = logp.exp_()
            dz.add_(p, alpha=1 - alpha)
            mass.add_(p, alpha=1 - alpha)
            dz.scatter_add_(1, y, torch.full_like(y, -(1 - alpha), dtype=torch.float64))
            e_loss += (1 - alpha) * e
            del p, logp
        if soft:
            j = x["indices"][r][k]
            logq = torch.log_softmax(x["teacher"][r][k].double() / tau, 1)
            logp = torch.log_softmax(z / tau, 1)
            loss += alpha * tau ** 2 * (logq.exp() * (logq - logp.gather(1, j))).sum(1)
            p = logp.exp_()
            dz.add_(p, alpha=alpha * tau)
            dz.scatter_add_(1, j, -alpha * tau * logq.exp())
            mass.add_(p, alpha=alpha * tau)
            mass.scatter_add_(1, j, alpha * tau * logq.exp())
            e_loss += alpha * tau ** 2 * (e + float(logq.abs().max()) * 2.0 ** -21)
            del p, logp
        got = out["token_losses"][r][k].double()
        assert float((got - loss).abs().max()) <= e_loss + float(loss.max()) * 2.0 ** -22
        total += float(loss.sum())
        dz *= s
        err = mass.mul_(abs(s) * e).add_(dz.abs(), alpha=bits)
        gh = dz @ w
        eh = err @ w.abs() + (dz.abs() @ w.abs()) * (sum_steps(dtype, vocab) + 2.0 ** -18) + gh.abs() * half_step(dtype)
        off = (out["gh"][r][k].double() - gh).abs()
        assert bool((off <= eh).all()), (r, a, float((off / eh).max()))
        gw += dz.t() @ h
        ew += err.t() @ h.abs() + (dz.abs().t() @ h.abs()) * (sum_steps(dtype, len(keep)) + 2.0 ** -22)
        del z, dz, err, mass
    skipped = x["targets"][r] == IGNORE
    assert bool((out["gh"][r][skipped] == 0).all()) and bool((out["token_losses"][r][skipped] == 0).all())
    gw += old[r].double() if old is not None else 0.0
    ew += gw.abs() * half_step(dtype) * (2 if old is not None else 1)
    off = (out["gw"][r].double() - gw).abs()
    assert bool((off <= ew + 1e-37).all()), (r, float((off / (ew + 1e-37)).max()))
    assert abs(float(out["loss"][r]) - total * f) <= f * len(keep) * e_loss + abs(total * f) * 2.0 ** -22


def _call(x, how, dtype, accumulate, scale, alpha, tau, entries):
    out = dict(token_losses=[torch.full((h.shape[0],), float("nan"), device="cuda") for h in x["hidden"]],
               gh=[torch.full_like(h, float("nan")) for h in x["hidden"]], gw=[torch.full_like(w, float("nan")) for w in x["weights"]])
    old = None
    if accumulate:
        gen = torch.Generator(device="cuda").manual_seed(99)
        old = [(torch.randn(w.shape, device="cuda", generator=gen) * 1e-3).to(dtype) for w in x["weights"]]
        for g, o in zip(out["gw"], old):
            g.copy_(o)
    head = ddp.LossHead(x["weights"], out["gw"], max_tokens=max(max(h.shape[0] for h in x["hidden"]), 1), max_teacher=entries)
    head._workspace.fill_(255)
    args = dict(reduction=how, scale=scale, accumulate=accumulate, token_losses=out["token_losses"])
    if alpha > 0:
        out["loss"] = head.distill_grad(x["hidden"], x["teacher"], x["indices"], out["gh"], targets=x["targets"], alpha=alpha,
                                        temperature=tau, **args)
    else:
        out["loss"] = head.cross_entropy_grad(x["hidden"], x["targets"], out["gh"], **args)
    torch.cuda.synchronize()
    assert ddp.ddp_device_status() == 0
    return out, old


def _inputs(tokens, vocab, dim, dtype, seed, entries=0, edges=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(device="cuda", generator=gen)
    x = dict(weights=[], hidden=[], targets=[], teacher=[], indices=[])
    for n in tokens:
        x["weights"].append((torch.randn(vocab, dim, **kw) * dim ** -0.5).to(dtype))
        x["hidden"].append(torch.randn(n, dim, **kw).to(dtype))
        y = torch.randint(0, vocab, (n,), **kw)
        if edges:                                       # where a piece may begin, and the column before it
            y = torch.where(torch.rand(n, **kw) < 0.5, (y // 256 * 256 - torch.randint(0, 2, (n,), **kw)).clamp(min=0), y)
        y[torch.rand(n, **kw) < 0.1] = IGNORE
        x["targets"].append(y)
        if entries:
            # distinct: one of each run of columns, half of them at its edges
            run = vocab // entries // 256 * 256 if edges else vocab // entries
            first = torch.arange(entries, device="cuda") * run
            j = first + torch.randint(0, run, (n, entries), **kw)
            if edges:
                j = torch.where(torch.rand(n, entries, **kw) < 0.5, j // 256 * 256 + 255 * torch.randint(0, 2, (n, entries), **kw), j)
            x["indices"].append(j)
            x["teacher"].append(torch.randn(n, entries, **kw) * 2)
    return x


@TYPES
@pytest.mark.parametrize("op,alpha,tau", [("ce", 0.0, 1.0), ("distill", 0.5, 2.0), ("distill", 1.0, 2.0), ("distill", 0.25, 1.0)])
def test_pieces_of_two_ranks(dtype, op, alpha, tau):
    # 16-bit exponentials of 8448 rows by 131200 columns take 2.07 GiB, float32's of 2048 rows 2.5: so neither is kept, and
    # the pieces' logits are computed again; the second rank is shorter
    tokens, vocab, dim = ([8300, 1500] if dtype == BF16 else [2000, 700]), 131200, 16
    x = _inputs(tokens, vocab, dim, dtype, seed=31, entries=12 if alpha > 0 else 0, edges=True)
    for accumulate, how in ((False, ddp.DDP_LOSS_MEAN), (True, ddp.DDP_LOSS_WORLD_MEAN)):
        out, old = _call(x, how, dtype, accumulate, 2.0, alpha, tau, 12 if alpha > 0 else 0)
        counts = [int((t != IGNORE).sum()) for t in x["targets"]]
        for r in range(2):
            f = 1.0 / counts[r] if how == ddp.DDP_LOSS_MEAN else 2.0 / sum(counts)
            _check_rank(x, r, out, f, 2.0, alpha, tau, old)


@TYPES
@pytest.mark.parametrize("dim", [130, 128, 1])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("alpha,tau", [(0.0, 1.0), (0.5, 3.0)])
def test_a_depth_of_several_parts(dtype, dim, accumulate, alpha, tau):
    # float32 takes 1024 rows of a rank, and 1024 columns of the vocabulary, at a time
    tokens, vocab = [3333, 1025], 2500
    x = _inputs(tokens, vocab, dim, dtype, seed=32, entries=7 if alpha > 0 else 0)
    out, old = _call(x, ddp.DDP_LOSS_SUM, dtype, accumulate, 1.0, alpha, tau, 7 if alpha > 0 else 0)
    for r in range(2):
        _check_rank(x, r, out, 1.0, 1.0, alpha, tau, old)


@TYPES
@pytest.mark.parametrize("tokens", [[0, 0], [0], [0] * 16 + [3, 2], [3] * 16 + [0, 0]])
@pytest.mark.parametrize("vocab,dim", [(100, 32), (777, 128)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_ranks_without_tokens(dtype, tokens, vocab, dim, accumulate):
    x = _inputs(tokens, vocab, dim, dtype, seed=33, entries=4)
    out, old = _call(x, ddp.DDP_LOSS_WORLD_MEAN, dtype, accumulate, 1.0, 0.0, 1.0, 4)
    for r, n in enumerate(tokens):
        if n == 0:
            assert float(out["loss"][r]) == 0.0
            assert torch.equal(out["gw"][r], old[r] if accumulate else torch.zeros_like(out["gw"][r]))
        else:
            f = len(tokens) / max(sum(int((t != IGNORE).sum()) for t in x["targets"]), 1)
            _check_rank(x, r, out, f, 1.0, 0.0, 1.0, old)


@TYPES
@pytest.mark.parametrize("tau", [0.25, 0.5, 2.0, 4.0, 5.0])
@pytest.mark.parametrize("tokens,vocab,dim", [(64, 3000, 64), (16, 100, 32)])
def test_logits_gradients_of_two_temperatures(dtype, tau, tokens, vocab, dim):
    """Each logit's gradient for itself: hidden states that are unit vectors make the weights' gradients the logits'.

    Columns that nobody lists are sums of two softmaxes, so their relative errors do not add up beyond the larger:
    exponents of up to 9 at most times 1 / tau, three roundings each, an exponential's and two sums' steps; in bf16 the
    kept exponential's 2^-11, times max(tau, 1 / tau) up to 4 for the steeper one (beyond 4 nothing is kept), and bf16's
    2^-8."""
    x = _inputs([tokens], vocab, dim, dtype, seed=34, entries=5)
    x["weights"][0] = (torch.randn(vocab, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(35)).clamp(-4, 4)).to(dtype)
    x["hidden"][0] = torch.eye(tokens, dim, device="cuda").to(dtype)
    x["targets"][0] = x["targets"][0].clamp(min=0)
    out, _ = _call(x, ddp.DDP_LOSS_SUM, dtype, False, 1.0, 0.5, tau, 5)
    z = x["weights"][0].double().t()[:tokens]
    p, pt = torch.softmax(z, 1), torch.softmax(z / tau, 1)
    dz = 0.5 * p + 0.5 * tau * pt
    got = out["gw"][0].double().t()[:tokens]
    listed = torch.zeros_like(z, dtype=torch.bool).scatter(1, x["indices"][0], True).scatter(1, x["targets"][0].unsqueeze(1), True)
    sharp = max(1.0, 1 / tau)
    rel = 9 * sharp * (3 * 2.0 ** -24 + 1.6e-8 * dim / 16 + 2.0 ** -24) + 4 * 2.0 ** -22 + 2 * 64 * 2.0 ** -24
    rel += max(tau, 1 / tau) * 2.0 ** -11 + 2.0 ** -8 if dtype == BF16 else max(tau, 1 / tau) * 2.0 ** -21 + 2.0 ** -18
    assert float(((got - dz).abs() / dz)[~listed].max()) <= rel
    # the listed ones, whose parts may cancel: float32 steps of the parts, and the result's rounding
    q = torch.softmax(x["teacher"][0].double() / tau, 1)
    mass = dz.scatter_add(1, x["indices"][0], 0.5 * tau * q) + torch.zeros_like(z).scatter(1, x["targets"][0].unsqueeze(1), 0.5)
    dz = dz.scatter_add(1, x["indices"][0], -0.5 * tau * q).scatter_add(1, x["targets"][0].unsqueeze(1), torch.full_like(z[:, :1], -0.5))
    bound = mass * (9 * sharp * 2.0 ** -21 + 2.0 ** -19) + dz.abs() * (2.0 ** -8 if dtype == BF16 else 2.0 ** -18)
    assert bool(((got - dz).abs() <= bound)[listed].all())
