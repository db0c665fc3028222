"""The loss head's definition in float64, and how far float32 and bf16 arithmetic may be from it.

Bounds, all of them products of half steps (eps / 2: bf16 2^-8, float32 2^-24) with sums of magnitudes:
  * a logit is a sum of products of bf16 values, exact in float32, or of three-part splits whose omitted products are
    below 4 x 2^-24 of the terms; the tensor cores add 16 products at a time and may cut instead of rounding, so each step is off by
    2^-23 of the magnitudes' sum at most;
  * exponentials and logarithms are off by 2^-21 relative, arguments of size a by a x 2^-23;
  * the logits' gradients are rounded to bf16 (or split in three parts) for their products, sums as above;
  * results are rounded once to their type.
"""
import torch

IGNORE = -100
LOSS = {"sum": 0, "mean": 1, "world_mean": 2}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sum_steps(dtype, depth):
    """Relative to the magnitudes' sum: steps of 16 products, six passes over three-part operands."""
    f32 = dtype == torch.float32
    return ((6 if f32 else 1) * -(-depth // 16) + 16) * 2.0 ** -23 + (4 * 2.0 ** -24 if f32 else 0.0)


def reference(hidden, weights, targets=None, teacher=None, indices=None, temperature=1.0, alpha=None, reduction="mean", ignore=IGNORE,
              scale=1.0, columns_of=None):
    """Everything of a call in float64 on the tensors' device, with bounds: a list of dicts, one a rank."""
    world, distill = len(hidden), teacher is not None
    alpha = (1.0 if distill else 0.0) if alpha is None else alpha
    keep = []
    for r in range(world):
        ok = torch.ones(hidden[r].shape[0], dtype=torch.bool, device=hidden[r].device)
        if targets is not None:
            ok &= (targets[r] != ignore) & (targets[r] >= 0) & (targets[r] < weights[r].shape[0])
        if distill:
            there = (indices[r] >= 0) & (indices[r] < weights[r].shape[0]) & (teacher[r] != -float("inf"))
            ok &= there.any(1)
        keep.append(ok)
    total = sum(int(k.sum()) for k in keep)
    out = []
    for r in range(world):
        dtype, device, ok = weights[r].dtype, weights[r].device, keep[r]
        n = int(ok.sum())
        f = {"sum": 1.0, "mean": 1.0 / max(n, 1), "world_mean": world / max(total, 1)}[reduction]
        h, w = hidden[r][ok].double(), weights[r].double()
        vocab, dim = w.shape
        z = h @ w.t()
        size = (h.abs() @ w.abs().t())
        dz_logit = float(size.max() * sum_steps(dtype, dim)) if n else 0.0
        big = float(z.abs().max()) if n else 0.0
        loss = torch.zeros(n, dtype=torch.float64, device=device)
        g = torch.zeros_like(z)
        mass = torch.zeros_like(z)                       # what the softmaxes' relative errors multiply
        e_exp = 2 * dz_logit + (big + 40) * 2.0 ** -21
        e_loss = 0.0
        if alpha < 1.0:
            y = targets[r][ok].unsqueeze(1)
            logp = torch.log_softmax(z, 1)
            loss += (1 - alpha) * -logp.gather(1, y).squeeze(1)
            p = logp.exp()
            g += (1 - alpha) * p
            mass += (1 - alpha) * p
            g.scatter_add_(1, y, torch.full_like(y, -(1 - alpha), dtype=torch.float64))
            e_loss += (1 - alpha) * e_exp
        if distill:
            there = (indices[r][ok] >= 0) & (indices[r][ok] < vocab) & (teacher[r][ok] != -float("inf"))
            col = torch.where(there, indices[r][ok], torch.zeros_like(indices[r][ok]))
            t = (teacher[r][ok].double() / temperature).masked_fill(~there, -float("inf"))
            q = torch.softmax(t, 1)
            logq = torch.log_softmax(t, 1)
            logp = torch.log_softmax(z / temperature, 1)
            terms = q * (logq - logp.gather(1, col))
            loss += alpha * temperature ** 2 * torch.where(q > 0, terms, torch.zeros_like(terms)).sum(1)
            p = logp.exp()
            g += alpha * temperature * p
            g.scatter_add_(1, col, -alpha * temperature * q)
            mass += alpha * temperature * p
            mass.scatter_add_(1, col, alpha * temperature * q)
            e_exp = e_exp * max(1.0, 1 / temperature) + float(t[there].abs().max() if there.any() else 0) * 2.0 ** -21
            e_loss += alpha * temperature ** 2 * e_exp
        full = torch.zeros(hidden[r].shape[0], dtype=torch.float64, device=device)
        full[ok] = loss
        s = abs(scale) * f
        dz = g * f * scale
        # of a logit's gradient: the softmaxes' errors, and its rounding for the products
        err = mass * s * e_exp + dz.abs() * (half_step(torch.bfloat16) if dtype == torch.bfloat16 else 2.0 ** -23)
        gh, gw = dz @ w, dz.t() @ h
        eh = err @ w.abs() + (dz.abs() @ w.abs()) * (sum_steps(dtype, vocab) + 2.0 ** -18) + gh.abs() * half_step(dtype)
        ew = err.t() @ h.abs() + (dz.abs().t() @ h.abs()) * (sum_steps(dtype, max(n, 1)) + 2.0 ** -22) + gw.abs() * half_step(dtype)
        grad_hidden = torch.zeros(hidden[r].shape, dtype=torch.float64, device=device)
        hidden_bound = torch.zeros_like(grad_hidden)
        grad_hidden[ok], hidden_bound[ok] = gh, eh
        out.append(dict(n=n, token_losses=full, token_bound=e_loss + full.abs().max().item() * 2.0 ** -22 if n else 0.0,
                        loss=float(loss.sum() * f), loss_bound=f * n * e_loss + abs(float(loss.sum() * f)) * 2.0 ** -22,
                        grad_hidden=grad_hidden, hidden_bound=hidden_bound, grad_weights=gw, weights_bound=ew))
    return out


def check(want, loss, token_losses=None, grad_hidden=None, grad_weights=None):
    for r, x in enumerate(want):
        assert abs(float(loss[r]) - x["loss"]) <= x["loss_bound"], (r, float(loss[r]), x["loss"], x["loss_bound"])
        if token_losses is not None:
            off = (token_losses[r].double() - x["token_losses"]).abs().max().item() if x["token_losses"].numel() else 0.0
            assert off <= x["token_bound"], (r, off, x["token_bound"])
        for got, name, bound in ((grad_hidden, "grad_hidden", "hidden_bound"), (grad_weights, "grad_weights", "weights_bound")):
            if got is not None and x[name].numel():
                off = (got[r].double() - x[name]).abs()
                over = off > x[bound] + 1e-37
                assert not bool(over.any()), (r, name, int(over.sum()), float((off / (x[bound] + 1e-37)).max()))
                assert not bool(got[r].isnan().any()), (r, name)
