"""Cases of the loss head's operators: softmax cross entropy over a vocabulary without keeping its logits, and distillation
from a teacher's top logits, each as a loss alone and with its gradients, with their plain forms.

Every rank has its own copy of the head's weights and its own tokens; a rank's tokens may be fewer than another's.  The
weights' gradients are what a sync of the ranks' gradients takes.
"""
import math

import torch

own = False

IGNORE = -100
REDUCTIONS = {"sum": 0, "mean": 1, "world_mean": 2}      # as the framework numbers them


def _tokens(case):
    """Tokens of each rank; a case holds them as text."""
    return [int(n) for n in case["tokens"].split()]


TINY = dict(vocab=100, dim=32)
DECODER = dict(vocab=50257, dim=1024)


def listed():
    return [
        # the loss of one new token of the tiny decoder: the call's latency
        dict(TINY, name="ce_loss_one_token_bf16", op="ce_loss", dtype="bf16", tokens="1", ignored=0.0, reduction="sum"),
        # validation of the 355M decoder on one sequence: memory and products count alike
        dict(DECODER, name="ce_loss_decoder_bf16", op="ce_loss", dtype="bf16", tokens="1024", ignored=0.0, reduction="mean"),
        # the same in float32 on two ranks whose last batches are ragged
        dict(DECODER, name="ce_loss_decoder_f32_n2", op="ce_loss", dtype="f32", tokens="777 301", ignored=0.05,
             reduction="world_mean"),
        # a training step of the tiny decoder on 4 ranks: latency
        dict(TINY, name="ce_grad_small_bf16_n4", op="ce_grad", dtype="bf16", tokens="16 16 16 16", ignored=0.0, reduction="mean"),
        # the 355M decoder on 8 ranks, a sequence each
        dict(DECODER, name="ce_grad_decoder_bf16_n8", op="ce_grad", dtype="bf16", tokens=" ".join(["1024"] * 8), ignored=0.0,
             reduction="mean"),
        # fine tuning on one rank, where the prompts' tokens are not learned: over a third of 8192 tokens are ignored
        dict(DECODER, name="ce_grad_prompts_bf16", op="ce_grad", dtype="bf16", tokens="8192", ignored=0.35,
             reduction="mean"),
        # float32 weights and gradients, two ranks
        dict(DECODER, name="ce_grad_decoder_f32_n2", op="ce_grad", dtype="f32", tokens="1024 900", ignored=0.1,
             reduction="world_mean"),
        # odd sizes throughout: a small vocabulary, rows that no 16-byte boundary holds, ragged ranks
        dict(name="ce_grad_odd_bf16_n3", op="ce_grad", dtype="bf16", vocab=10007, dim=515, tokens="333 1 1025",
             ignored=0.2, reduction="world_mean"),
        # a large vocabulary and a wide model
        dict(name="ce_grad_large_bf16", op="ce_grad", dtype="bf16", vocab=131072, dim=4096, tokens="4096", ignored=0.0,
             reduction="mean"),
        # how far a student is from its teacher: one sequence, 32 logits a token
        dict(DECODER, name="distill_loss_decoder_bf16", op="distill_loss", dtype="bf16", tokens="1024", ignored=0.1,
             reduction="mean", teacher=32, temperature=1.0, alpha=1.0, targets=False),
        # a small student on 2 ranks: latency
        dict(TINY, name="distill_grad_small_f32_n2", op="distill_grad", dtype="f32", tokens="16 7", ignored=0.1,
             reduction="world_mean", teacher=8, temperature=2.0, alpha=0.5, targets=True),
        # training a student on 2 ranks, half from the labels and half from the teacher's 64 logits
        dict(DECODER, name="distill_grad_decoder_bf16_n2", op="distill_grad", dtype="bf16", tokens="2048 2048", ignored=0.1,
             reduction="world_mean", teacher=64, temperature=2.0, alpha=0.5, targets=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    while True:
        op = rng.choice(["ce_loss", "ce_grad", "distill_loss", "distill_grad"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        world = rng.choice([1, 1, 2, 3, 4, 8])
        longest = _log_int(rng, 1, 8192)
        tokens = [longest] + [max(1, int(longest * rng.uniform(0.2, 1.0))) for _ in range(world - 1)]
        vocab, dim = _log_int(rng, 8, 131072), _log_int(rng, 8, 4096)
        if rng.random() < 0.5:                           # as models have them
            vocab, dim = -(-vocab // 8) * 8, -(-dim // 64) * 64
        # below the largest listed case, and in float32 below what takes the plain form as long
        if sum(tokens) * vocab * dim < (1e12 if dtype == "bf16" else 1.5e11) and world * vocab * dim < 6e8:
            break
    case = dict(op=op, dtype=dtype, vocab=vocab, dim=dim, tokens=" ".join(map(str, tokens)), ignored=rng.choice([0.0, 0.1, 0.5]),
                reduction=rng.choice(sorted(REDUCTIONS)))
    if op.startswith("distill"):
        targets = rng.random() < 0.5
        case.update(teacher=min(vocab, _log_int(rng, 1, 128)), temperature=rng.choice([1.0, 2.0, 3.5]), targets=targets,
                    alpha=rng.choice([0.25, 0.5, 0.9]) if targets else 1.0)
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    """Weights with logits of about unit spread, and hidden states that lean towards their target's row, by 0 to 12 in its
    logit, as a model that has learned some.  A teacher's entries are distinct columns, its logits fall with their rank and
    the first is mostly the target; the tokens that are not learned have no entries (index -1) where there are no
    targets to say so.  The framework's side also gets what a program makes once and keeps: the handle with its workspace,
    and the tensors that results go to."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    vocab, dim, tokens = case["vocab"], case["dim"], _tokens(case)
    world = len(tokens)
    rand = dict(device="cuda", generator=gen)
    first = (torch.randn(vocab, dim, **rand) * dim ** -0.5).to(dtype)
    x = dict(case, tokens=tokens, weights=[first] + [first.clone() for _ in range(world - 1)], hidden=[], labels=[])
    distill = case["op"].startswith("distill")
    if distill:
        x.update(logits=[], indices=[])
    for n in tokens:
        y = torch.randint(0, vocab, (n,), **rand)
        lean = torch.rand(n, 1, **rand) * 12.0
        x["hidden"].append((torch.randn(n, dim, **rand) + lean * first[y].float()).to(dtype))
        skip = torch.rand(n, **rand) < case["ignored"]
        if distill:
            k = case["teacher"]
            gaps = torch.randint(1, vocab // k + 1, (n, k), **rand)
            gaps[:, 0] = 0                               # the first entry is the target
            order = torch.rand(n, k, **rand)
            order[:, 0] = -1.0
            columns = ((y.unsqueeze(1) + gaps.cumsum(1)) % vocab).gather(1, order.argsort(1))
            rank = torch.arange(1, k + 1, device="cuda").log()
            x["logits"].append(9.0 - 2.0 * rank + 0.5 * torch.randn(n, k, **rand))
            if not case["targets"]:
                columns[skip] = -1
            x["indices"].append(columns)
        x["labels"].append(y.masked_fill(skip, IGNORE))
    if own:
        import gradient_sync_plan_gb300 as ddp
        grads = case["op"].endswith("grad")
        x["grad_weights"] = [torch.empty_like(w) for w in x["weights"]] if grads else None
        x["grad_hidden"] = [torch.empty_like(h) for h in x["hidden"]] if grads else None
        x["token_losses"] = [torch.empty(n, device="cuda") for n in tokens]
        x["head"] = ddp.LossHead(x["weights"], x["grad_weights"], max_tokens=max(tokens),
                                 max_teacher=case["teacher"] if distill else 0)
    return x


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _lse(z):
    top = z.max(dim=1, keepdim=True).values
    return (z - top).exp().sum(dim=1, keepdim=True).log() + top


def _valid(x, r):
    if x["op"].startswith("distill") and not x["targets"]:
        return (x["indices"][r] >= 0).any(dim=1)
    return x["labels"][r] != IGNORE


def _factor(x, counts, r):
    """What rank r's sum of token losses is multiplied by."""
    if x["reduction"] == "sum":
        return torch.ones((), device="cuda")
    if x["reduction"] == "mean":
        return 1.0 / counts[r].clamp(min=1).float()
    return len(counts) / torch.stack(counts).sum().clamp(min=1).float()


def _plain_rank(x, r, factor, grad):
    valid = _valid(x, r).unsqueeze(1)
    h, w = x["hidden"][r].float(), x["weights"][r].float()
    z = h @ w.t()
    lse = _lse(z)
    distill = x["op"].startswith("distill")
    alpha, tau = (x["alpha"], x["temperature"]) if distill else (0.0, 1.0)
    rows = torch.arange(h.shape[0], device="cuda")
    y = x["labels"][r].clamp(min=0)
    loss = torch.zeros_like(lse)
    if alpha < 1.0:
        loss += (1.0 - alpha) * (lse - z.gather(1, y.unsqueeze(1)))
    if distill:
        columns = x["indices"][r].clamp(min=0)
        lse_tau = _lse(z / tau)
        log_q = x["logits"][r] / tau
        log_q = log_q - _lse(log_q)
        q = log_q.exp()
        loss += alpha * tau * tau * (q * (log_q - z.gather(1, columns) / tau + lse_tau)).sum(dim=1, keepdim=True)
    loss = torch.where(valid, loss, torch.zeros_like(loss)).squeeze(1)
    if not grad:
        return loss, None, None
    if distill:
        dz = (z / tau - lse_tau).exp().mul_(alpha * tau)
        dz.scatter_add_(1, columns, q * (-alpha * tau))
        if alpha < 1.0:
            dz += (z - lse).exp_().mul_(1.0 - alpha)
            dz[rows, y] -= 1.0 - alpha
    else:
        dz = (z - lse).exp_()
        dz[rows, y] -= 1.0
    del z
    dz.mul_(valid * factor)
    dtype = x["hidden"][r].dtype
    return loss, (dz @ w).to(dtype), (dz.t() @ h).to(dtype)


def _plain(x, grad):
    world = len(x["tokens"])
    counts = [_valid(x, r).sum() for r in range(world)]
    out = dict(loss=[], token_losses=[], grad_hidden=[], grad_weights=[])
    for r in range(world):
        factor = _factor(x, counts, r)
        loss, gh, gw = _plain_rank(x, r, factor, grad)
        out["loss"].append(loss.sum() * factor)
        out["token_losses"].append(loss)
        out["grad_hidden"].append(gh)
        out["grad_weights"].append(gw)
    out["loss"] = torch.stack(out["loss"])
    return out if grad else {k: out[k] for k in ("loss", "token_losses")}


def run(state):
    x = state
    grad = x["op"].endswith("grad")
    if not own:
        return _plain(x, grad)
    head = x["head"]
    how = dict(reduction=REDUCTIONS[x["reduction"]], ignore_index=IGNORE, token_losses=x["token_losses"])
    if x["op"] == "ce_loss":
        loss = head.cross_entropy(x["hidden"], x["labels"], **how)
    elif x["op"] == "ce_grad":
        loss = head.cross_entropy_grad(x["hidden"], x["labels"], x["grad_hidden"], **how)
    else:
        how.update(targets=x["labels"] if x["targets"] else None, alpha=x["alpha"], temperature=x["temperature"])
        if grad:
            loss = head.distill_grad(x["hidden"], x["logits"], x["indices"], x["grad_hidden"], **how)
        else:
            loss = head.distill(x["hidden"], x["logits"], x["indices"], **how)
    out = dict(loss=loss, token_losses=x["token_losses"])
    return dict(out, grad_hidden=x["grad_hidden"], grad_weights=x["grad_weights"]) if grad else out


# ---------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    """The tokens that are learned count for the products, on average; the gradients take two products beside the
    logits'."""
    size = 2 if case["dtype"] == "bf16" else 4
    grad = case["op"].endswith("grad")
    tokens, world = sum(_tokens(case)), len(_tokens(case))
    learned = max(1.0, tokens * (1.0 - case["ignored"]))
    matrices = (world * case["vocab"] + tokens) * case["dim"] * size * (2 if grad else 1)
    labels = 12 * tokens + (12 * tokens * case["teacher"] if case["op"].startswith("distill") else 0)
    return {"bytes": float(matrices + labels), "flops": (6.0 if grad else 2.0) * learned * case["vocab"] * case["dim"]}


def exact(case, seed):
    """Rank by rank in float64, on the learned tokens' rows alone."""
    x = prepare(case, seed)
    grad, distill = case["op"].endswith("grad"), case["op"].startswith("distill")
    tokens = _tokens(case)
    world = len(tokens)
    hard = not distill or case["targets"]
    kept = [(x["labels"][r] != IGNORE if hard else (x["indices"][r] >= 0).all(1)).nonzero()[:, 0] for r in range(world)]
    total = sum(len(k) for k in kept)
    out = dict(loss=[], token_losses=[], grad_hidden=[], grad_weights=[])
    for r, keep in enumerate(kept):
        f = {"sum": 1.0, "mean": 1.0 / max(1, len(keep)), "world_mean": world / max(1, total)}[case["reduction"]]
        h, w = x["hidden"][r][keep].double(), x["weights"][r].double()
        z = torch.mm(h, w.transpose(0, 1))
        losses = torch.zeros(len(keep), dtype=torch.float64, device="cuda")
        d = torch.zeros_like(z) if grad else None
        if hard:
            part = 1.0 - case["alpha"] if distill else 1.0
            y = x["labels"][r][keep]
            logp = torch.log_softmax(z, 1)
            losses -= part * logp.gather(1, y[:, None])[:, 0]
            if grad:
                logp.exp_()
                logp.scatter_add_(1, y[:, None], -torch.ones_like(losses)[:, None])
                d += part * f * logp
            del logp
        if distill:
            tau, a = case["temperature"], case["alpha"]
            logp = torch.log_softmax(z / tau, 1)
            q = torch.log_softmax(x["logits"][r][keep].double() / tau, 1)
            columns = x["indices"][r][keep]
            losses += a * tau ** 2 * (q.exp() * (q - logp.gather(1, columns))).sum(1)
            if grad:
                d += a * tau * f * logp.exp_()
                d.scatter_add_(1, columns, -a * tau * f * q.exp())
            del logp
        full = torch.zeros(tokens[r], dtype=torch.float64, device="cuda")
        full[keep] = losses
        out["loss"].append(losses.sum() * f)
        out["token_losses"].append(full)
        if grad:
            gh = torch.zeros(tokens[r], case["dim"], dtype=torch.float64, device="cuda")
            gh[keep] = torch.mm(d, w)
            out["grad_hidden"].append(gh)
            out["grad_weights"].append(torch.mm(d.transpose(0, 1), h))
    out["loss"] = torch.stack(out["loss"])
    return out if grad else {k: out[k] for k in ("loss", "token_losses")}
