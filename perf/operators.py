"""Cases of the gradient norm, clipping, norm-in-the-sync and AdamW operators, with their plain forms.

Each rank's tensors are views into one row of a [world, row] storage, either "packed" back to back (the gradients are
views into a flat bucket, so most tensors start at odd addresses) or "apart", each on a boundary of 256 elements as an allocator
places them, with zeros between.  The plain forms compute on the storage as a whole.
"""
import math
import random

import torch

own = False

EPS_CLIP = 1e-6
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1


# ---------------------------------------------------------------------------
# Parameter lists
# ---------------------------------------------------------------------------

def _decoder(layers, d, ff, vocab, pos):
    layer = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, d * ff, ff, ff * d, d]
    return [vocab * d, pos * d] + layer * layers + [d, d]


def _resnet50():
    def block(i, planes, cin):
        body = [planes * cin, planes, planes, 9 * planes * planes, planes, planes, 4 * planes * planes, 4 * planes,
                4 * planes]
        return body + ([4 * planes * cin, 4 * planes, 4 * planes] if i == 0 else [])
    stages = [(64, 3, 64), (128, 4, 256), (256, 6, 512), (512, 3, 1024)]
    return [64 * 3 * 49, 64, 64] + [x for planes, n, cin in stages for i in range(n)
                                    for x in block(i, planes, cin if i == 0 else 4 * planes)] + [1000 * 2048, 1000]


def _split(total, tensors, seed):
    """`tensors` sizes of at least one element that add up to `total`, over several orders of magnitude."""
    r = random.Random(seed)
    w = [math.exp(r.gauss(0.0, 2.0)) for _ in range(tensors)]
    sizes = [1 + int((total - tensors) * x / sum(w)) for x in w]
    return sizes[:-1] + [total - sum(sizes[:-1])]


def _numels(case):
    if case["params"] == "decoder":
        return _decoder(case["layers"], case["d"], case["ff"], case["vocab"], case["pos"])
    if case["params"] == "resnet50":
        return _resnet50()
    return _split(case["total"], case["tensors"], case["split"])


def _offsets(case, numels):
    """Element offset of each tensor in its row, and the row's length (a multiple of 256 elements)."""
    step = 256 if case["layout"] == "apart" else 1
    ends = torch.tensor([-(-n // step) * step for n in numels], dtype=torch.int64).cumsum(0).tolist()
    return [0] + ends[:-1], -(-ends[-1] // 256) * 256


SMALL = dict(params="decoder", layers=2, d=32, ff=64, vocab=100, pos=16)
MEDIUM = dict(params="resnet50")
LARGE = dict(params="decoder", layers=24, d=1024, ff=4096, vocab=50257, pos=1024)


def listed():
    return [
        # the norm of one rank's gradients: a tiny decoder, where the call's latency counts
        dict(SMALL, name="norm_small_f32", op="norm", dtype="f32", world=1, layout="apart"),
        # ResNet-50's bf16 gradients on one rank: 161 tensors, 51 MB
        dict(MEDIUM, name="norm_resnet50_bf16", op="norm", dtype="bf16", world=1, layout="apart"),
        # every rank's own norm before a sync: the 355M decoder on 8 ranks, gradients as bucket views
        dict(LARGE, name="norm_decoder_f32_n8", op="norm", dtype="f32", world=8, layout="packed"),
        # scaling by a norm that is already known, as after a sync that returned it: the tiny decoder
        dict(SMALL, name="clip_small_f32", op="clip", dtype="f32", world=1, layout="packed"),
        # ResNet-50's gradients on two ranks, separate allocations
        dict(MEDIUM, name="clip_resnet50_f32_n2", op="clip", dtype="f32", world=2, layout="apart"),
        # the 355M decoder's bf16 gradients on four ranks
        dict(LARGE, name="clip_decoder_bf16_n4", op="clip", dtype="bf16", world=4, layout="apart"),
        # the whole sync of a tiny decoder on 4 ranks, with the averaged gradient's norm
        dict(SMALL, name="sync_norm_small_f32_n4", op="sync_norm", dtype="f32", world=4, layout="apart"),
        # ResNet-50 on 2 ranks: the norm's own pass would be a fifth of the traffic
        dict(MEDIUM, name="sync_norm_resnet50_f32_n2", op="sync_norm", dtype="f32", world=2, layout="apart"),
        # the 355M decoder's step on 8 ranks
        dict(LARGE, name="sync_norm_decoder_f32_n8", op="sync_norm", dtype="f32", world=8, layout="apart"),
        # the update of a tiny decoder, fp32 throughout
        dict(SMALL, name="adamw_small_f32", op="adamw", dtype="f32", world=1, layout="apart", copies=False, t0=0),
        # mixed precision: bf16 gradients, fp32 weights and moments, bf16 weights written for the next forward
        dict(MEDIUM, name="adamw_resnet50_bf16_copies", op="adamw", dtype="bf16", world=1, layout="apart", copies=True,
             t0=100),
        # the 355M decoder's update on 2 ranks, flat fp32 buffers
        dict(LARGE, name="adamw_decoder_f32_n2", op="adamw", dtype="f32", world=2, layout="packed", copies=False,
             t0=20000),
    ]


def draw(rng):
    op = rng.choice(["norm", "clip", "sync_norm", "adamw"])
    world = rng.choice([1, 2, 3, 4, 5, 8, 13, 16]) if op != "sync_norm" else rng.choice([2, 3, 4, 5, 8, 13, 16])
    most = 6e8 if op == "adamw" else 2.5e9          # elements over all ranks, below the largest listed cases
    total = int(math.exp(rng.uniform(math.log(1.5e3), math.log(most / world))))
    case = dict(op=op, params="split", total=total, tensors=rng.randint(1, min(400, total)), split=rng.randrange(1 << 30),
                dtype="f32" if op == "sync_norm" else rng.choice(["f32", "bf16"]), world=world,
                layout=rng.choice(["packed", "apart"]))
    if op == "adamw":
        case.update(copies=rng.random() < 0.5, t0=rng.choice([0, 7, 1000]))
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _views(x, kind):
    return [[row[o:o + n] for n, o in zip(x["numels"], x["offsets"])] for row in x[kind]]


def prepare(case, seed):
    """The storage of each kind of tensor, from the seed: gradients whose size differs from tensor to tensor, a third of
    the larger ones with rows of zeros (embedding rows that no token used), and for the update weights and moments.
    The framework's side also gets what a program makes once and keeps: the tables of its tensors."""
    numels = _numels(case)
    offsets, row = _offsets(case, numels)
    world = case["world"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    grads = torch.zeros(world, row, dtype=dtype, device="cuda")
    for n, o in zip(numels, offsets):
        g = grads[:, o:o + n]
        g.normal_(0.0, 10.0 ** r.uniform(-4.0, -1.5), generator=gen)
        if n >= 4096 and r.random() < 0.33:
            g[:, n // 3:n // 2] = 0.0
    x = {"op": case["op"], "grads": grads, "numels": numels, "offsets": offsets}
    if case["op"] in ("clip", "adamw"):
        x["norms"] = torch.empty(world, device="cuda").uniform_(1.02, 1.5, generator=gen)
        x["max_norm"] = 1.0
    if case["op"] == "adamw":
        for kind, std in (("params", 2e-2), ("exp_avg", 1e-3), ("exp_avg_sq", 1e-3)):
            t = torch.zeros(world, row, device="cuda")
            if kind == "params" or case["t0"]:
                for n, o in zip(numels, offsets):
                    t[:, o:o + n].normal_(0.0, std, generator=gen)
            x[kind] = t.square_() if kind == "exp_avg_sq" else t
        x["copies"] = torch.zeros(world, row, dtype=torch.bfloat16, device="cuda") if case["copies"] else None
        x["steps"] = torch.full((world,), case["t0"], dtype=torch.int32, device="cuda")
    if own:
        import gradient_sync_plan_gb300 as ddp
        if case["op"] in ("norm", "clip"):
            x["set"] = ddp.GradSet(_views(x, "grads"))
        elif case["op"] == "sync_norm":
            plan = ddp.ddp_plan_buckets(numels, ddp.F32)
            x["call"] = ddp.SyncNormCall(_views(x, "grads"), plan, algo=ddp.DDP_ALGO_VIEW)
        else:
            x["opt"] = ddp.AdamW(_views(x, "params"), _views(x, "grads"), _views(x, "exp_avg"), _views(x, "exp_avg_sq"),
                                 copies=_views(x, "copies") if case["copies"] else None, steps=x["steps"])
    return x


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _plain_norm(g):
    return g.float().square().sum(dim=1).sqrt()


def _plain_scale(x):
    return (x["max_norm"] / (x["norms"] + EPS_CLIP)).clamp(max=1.0).unsqueeze(1)


def _plain_sync(x):
    g = x["grads"]
    mean = g.float().sum(dim=0) / g.shape[0]
    g.copy_(mean.to(g.dtype).expand_as(g))
    return _plain_norm(g[:1]).expand(g.shape[0])


def _plain_adamw(x):
    x["steps"] += 1
    t = x["steps"].float().unsqueeze(1)
    p, m, v = x["params"], x["exp_avg"], x["exp_avg_sq"]
    g = x["grads"].float() * _plain_scale(x)
    m.mul_(BETA1).add_(g * (1.0 - BETA1))
    v.mul_(BETA2).add_(g * g * (1.0 - BETA2))
    step = (m / (1.0 - BETA1 ** t)) / ((v / (1.0 - BETA2 ** t)).sqrt() + EPS)
    p.mul_(1.0 - LR * DECAY).sub_(step * LR)
    if x["copies"] is not None:
        x["copies"].copy_(p)


def _adamw_outputs(x):
    out = {"params": x["params"], "exp_avg": x["exp_avg"], "exp_avg_sq": x["exp_avg_sq"], "steps": x["steps"]}
    return out if x["copies"] is None else dict(out, copies=x["copies"])


def run(state):
    x, op = state, state["op"]
    if op == "norm":
        return x["set"].norm() if own else _plain_norm(x["grads"])
    if op == "clip":
        if own:
            x["set"].clip(x["max_norm"], x["norms"])
        else:
            x["grads"].copy_(x["grads"].float() * _plain_scale(x))
        return x["grads"]
    if op == "sync_norm":
        return {"norms": x["call"]() if own else _plain_sync(x), "grads": x["grads"]}
    if own:
        x["opt"].step(LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, norms=x["norms"], max_norm=x["max_norm"])
    else:
        _plain_adamw(x)
    return _adamw_outputs(x)


# ---------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    n = float(case["world"]) * sum(_numels(case))
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        return {"bytes": n * size, "flops": 2 * n}
    if case["op"] == "clip":
        return {"bytes": 2 * n * size, "flops": n}
    if case["op"] == "sync_norm":
        return {"bytes": 2 * n * size, "flops": n + 3 * n / case["world"]}
    return {"bytes": n * (size + 24 + (2 if case["copies"] else 0)), "flops": 15 * n}


def exact(case, seed):
    """Tensor by tensor, rank by rank, in float64."""
    x = prepare(case, seed)
    g, spans = x["grads"], [(o, o + n) for n, o in zip(x["numels"], x["offsets"])]
    world, row = g.shape
    if case["op"] == "norm":
        return torch.tensor([math.sqrt(math.fsum(float(g[r, a:b].double().pow(2).sum()) for a, b in spans))
                             for r in range(world)], dtype=torch.float64)
    if case["op"] == "sync_norm":
        mean, squares = torch.zeros(row, dtype=torch.float64, device="cuda"), []
        for a, b in spans:
            for r in range(world):
                mean[a:b] += g[r, a:b].double()
            mean[a:b] /= world
            squares.append(float(mean[a:b].pow(2).sum()))
        norms = torch.full((world,), math.sqrt(math.fsum(squares)), dtype=torch.float64)
        return {"norms": norms, "grads": mean.expand(world, row)}
    c = [min(1.0, x["max_norm"] / (float(n) + EPS_CLIP)) for n in x["norms"]]
    if case["op"] == "clip":
        out = torch.zeros(world, row, dtype=torch.float64, device="cuda")
        for r in range(world):
            for a, b in spans:
                out[r, a:b] = g[r, a:b].double() * c[r]
        return out
    t = case["t0"] + 1
    out = {k: x[k].double() for k in ("params", "exp_avg", "exp_avg_sq")}
    for r in range(world):
        for a, b in spans:
            d = g[r, a:b].double() * c[r]
            p, m, v = (out[k][r, a:b] for k in ("params", "exp_avg", "exp_avg_sq"))
            m.copy_(BETA1 * m + (1 - BETA1) * d)
            v.copy_(BETA2 * v + (1 - BETA2) * d ** 2)
            root = torch.sqrt(v / -math.expm1(t * math.log(BETA2))) + EPS
            p.copy_(p - LR * (DECAY * p + m / -math.expm1(t * math.log(BETA1)) / root))
    if case["copies"]:
        out["copies"] = out["params"]
    return dict(out, steps=None)
