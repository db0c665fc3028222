"""Values that the loss head's arithmetic may lose: NaN and infinities among the logits, small losses of confident tokens."""
import pytest
import torch

import gradient_sync_plan_gb300 as ddp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF16, F32])
# one launch; the tensor cores' kernels, the last unit of 128 columns having one
SHAPES = pytest.mark.parametrize("tokens,vocab,dim", [([16, 7], 100, 32), ([130, 40], 769, 128)])


def _inputs(tokens, vocab, dim, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(device="cuda", generator=gen)
    return dict(weights=[(torch.randn(vocab, dim, **kw) * dim ** -0.5).to(dtype) for _ in tokens],
                hidden=[torch.randn(n, dim, **kw).to(dtype) for n in tokens],
                targets=[torch.randint(0, vocab, (n,), **kw) for n in tokens],
                indices=[torch.rand(n, vocab, **kw).argsort(1)[:, :6].contiguous() for n in tokens],
                teacher=[torch.randn(n, 6, **kw) for n in tokens])


def _outputs(x, grads=True):
    return dict(token_losses=[torch.zeros(h.shape[0], device="cuda") for h in x["hidden"]],
                gw=[torch.zeros_like(w) for w in x["weights"]] if grads else None,
                gh=[torch.zeros_like(h) for h in x["hidden"]])


def _run(x, op, grads=True, **kw):
    """The outputs of a call; op: "ce", or "distill" with two temperatures and the targets' share."""
    out = _outputs(x, grads)
    head = ddp.LossHead(x["weights"], out["gw"], max_tokens=max(h.shape[0] for h in x["hidden"]), max_teacher=6)
    kw = dict(token_losses=out["token_losses"], **kw)
    if op == "distill":
        kw.update(targets=x["targets"], temperature=2.0, alpha=0.5)
        args = (x["hidden"], x["teacher"], x["indices"])
        out["loss"] = head.distill_grad(*args, out["gh"], **kw) if grads else head.distill(*args, **kw)
    else:
        args = (x["hidden"], x["targets"])
        out["loss"] = head.cross_entropy_grad(*args, out["gh"], **kw) if grads else head.cross_entropy(*args, **kw)
    torch.cuda.synchronize()
    assert ddp.ddp_device_status() == 0
    return out


@SHAPES
@TYPES
@pytest.mark.parametrize("op", ["ce", "distill"])
@pytest.mark.parametrize("grads", [False, True])
@pytest.mark.parametrize("where", ["all", "unit", "last", "one"])
def test_nan_among_the_weights_makes_the_losses_nan(tokens, vocab, dim, dtype, op, grads, where):
    # a padded vocabulary that nobody initialised: all columns, a whole unit of 128, the one column of the last unit, one of
    # many; every token's softmax has them in its sum
    x = _inputs(tokens, vocab, dim, dtype, seed=1)
    rows = dict(all=slice(0, None), unit=slice(0, min(128, vocab - 1)), last=slice(vocab - 1, None), one=slice(3, 4))[where]
    x["weights"][0][rows] = float("nan")
    out = _run(x, op, grads)
    assert bool(out["loss"][0].isnan()) and bool(out["token_losses"][0].isnan().all())
    if grads:
        assert bool(out["gh"][0].isnan().all()) and bool(out["gw"][0].isnan().all())
    # the other rank's are numbers
    assert bool(out["loss"][1].isfinite()) and bool(out["token_losses"][1].isfinite().all())
    if grads:
        assert bool(out["gh"][1].isfinite().all()) and bool(out["gw"][1].isfinite().all())


@SHAPES
@TYPES
@pytest.mark.parametrize("op", ["ce", "distill"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_in_a_learned_token_is_its_own(tokens, vocab, dim, dtype, op, bad):
    # infinity: some logits are +infinity, whose softmax is infinity over infinity
    x = _inputs(tokens, vocab, dim, dtype, seed=2)
    x["hidden"][0][3] = bad
    out = _run(x, op)
    nan = out["token_losses"][0].isnan()
    assert bool(nan[3]) and int(nan.sum()) == 1 and bool(out["loss"][0].isnan())
    nan = out["gh"][0].isnan()
    assert bool(nan[3].all()) and int(nan.sum()) == dim
    assert bool(out["gw"][0].isnan().all())          # that token's part of every row
    assert bool(out["loss"][1].isfinite()) and bool(out["gw"][1].isfinite().all())


@pytest.mark.parametrize("tokens,vocab,dim", [([16], 100, 32), ([130], 769, 128)])
def test_logits_of_minus_infinity_have_no_share(tokens, vocab, dim):
    x = _inputs(tokens, vocab, dim, BF16, seed=3)
    x["hidden"][0][:, 0] = 1.0
    masked = list(range(0, 64)) + [vocab - 1] + (list(range(128, 256)) if vocab > 256 else [])
    x["weights"][0][masked, 0] = -float("inf")
    x["targets"][0][:] = 70
    out = _run(x, "ce", grads=False)
    keep = torch.ones(vocab, dtype=torch.bool, device="cuda")
    keep[masked] = False
    z = x["hidden"][0].double() @ x["weights"][0][keep].double().t()
    want = torch.logsumexp(z, 1) - z[:, 70 - 64]
    # a logit's sum of `dim` products, twice, and the exponentials' and logarithm's steps
    size = float((x["hidden"][0].double().abs() @ x["weights"][0][keep].double().abs().t()).max())
    bound = 2 * size * (dim // 16 + 16) * 2.0 ** -23 + 40 * 2.0 ** -21
    assert float((out["token_losses"][0].double() - want).abs().max()) <= bound


@pytest.mark.parametrize("tokens,vocab,dim", [([16], 100, 32), ([130], 769, 128)])
@pytest.mark.parametrize("op", ["ce", "distill"])
@pytest.mark.parametrize("level", [0.0, -200.0, 200.0])
def test_columns_of_minus_infinity_have_no_gradient(tokens, vocab, dim, op, level):
    # whole units of 128 columns among them, beside logits around `level`; every other column's gradient is as without them
    x = _inputs(tokens, vocab, dim, BF16, seed=3)
    x["hidden"][0][:, :2] = 1.0
    x["weights"][0][:, 1] = level
    masked = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    masked[:64] = True
    masked[128:384] = True
    masked[vocab - 1] = True
    kept = (~masked).nonzero()[:, 0]
    x["targets"][0] = kept[x["targets"][0] % len(kept)]
    x["indices"][0] = kept[(torch.arange(6, device="cuda") * 5 + x["targets"][0].unsqueeze(1)) % len(kept)].contiguous()
    column = torch.full((vocab,), -1, dtype=torch.int64, device="cuda")
    column[kept] = torch.arange(len(kept), device="cuda")
    small = dict(x, weights=[x["weights"][0][kept].contiguous()], targets=[column[x["targets"][0]]], indices=[column[x["indices"][0]]])
    x["weights"][0][masked, 0] = -float("inf")
    out, want = _run(x, op), _run(small, op)
    assert bool((out["gw"][0][masked] == 0).all())
    # the same sums in other units of 128: a binary32 step or few of the loss, and of a logit's gradient what bf16 rounds twice
    assert float((out["token_losses"][0] - want["token_losses"][0]).abs().max()) <= 2.0 ** -16
    a, b = out["gw"][0][kept].double(), want["gw"][0].double()
    h = x["hidden"][0].double().abs()
    bound = 2 * (2.0 ** -8 + 2.0 ** -10) * (h.sum(0) / tokens[0]) + 2 * 2.0 ** -8 * b.abs()
    assert bool(((a - b).abs() <= bound).all())


CONFIDENT = [(16, 100, 32), (100, 769, 128), (60, 5000, 64)]


def _confident(tokens, vocab, dim, dtype, top, seed):
    """Logits that are what they are: token t's hidden state is the t-th unit vector, so column t of the weights holds its
    logits, and column t of the weights' gradients its logits' gradients.  The target's is `top`, the others' 8 to 20 below;
    all are bf16 values.  Returns the inputs and the logits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(device="cuda", generator=gen)
    y = torch.randint(0, vocab, (tokens,), **kw)
    z = top - 8.0 - 4.0 * torch.randint(0, 3, (tokens, 1), **kw) - 4.0 * torch.randint(0, 2, (tokens, vocab), **kw)
    z.scatter_(1, y.unsqueeze(1), torch.full((tokens, 1), float(top), device="cuda"))
    weights = torch.zeros(vocab, dim, device="cuda")
    weights[:, :tokens] = z.t()
    x = dict(weights=[weights.to(dtype)], hidden=[torch.eye(tokens, dim, device="cuda").to(dtype)], targets=[y],
             indices=[y.unsqueeze(1).contiguous()], teacher=[torch.randn(tokens, 1, **kw)])
    return x, z.double()


@pytest.mark.parametrize("tokens,vocab,dim", CONFIDENT)
@TYPES
@pytest.mark.parametrize("top", [28, 100, 1000, -100])
@pytest.mark.parametrize("op", ["ce", "distill"])
def test_losses_of_confident_tokens_keep_their_digits(tokens, vocab, dim, dtype, top, op):
    """A target that leads by 8 to 20 has a loss of log(1 + rest), 1e-9 to 0.3, whatever its logit; the teacher's one entry is
    the target, so the distillation's part is the same at its temperature.

    Relative error of the rest: an exponent of up to 20 from three roundings (2^-24 each) and the logits' own scale for the
    tensor cores (1.6e-8 a 16 of the depth, itself rounded by 2^-24), an exponential's 2^-22, a sum's 2^-24 times its 64
    additions in a row at most; a logarithm adds 2^-22.  Gradients are 1 / (1 + rest) times that with one more exponential
    and, of bf16, two roundings: kept exponentials' 2^-11 (11 bits), times 2 for the steeper softmax's, and bf16's 2^-8."""
    x, z = _confident(tokens, vocab, dim, dtype, top, seed=4)
    out = _run(x, op, reduction=ddp.DDP_LOSS_SUM)
    y = x["targets"][0].unsqueeze(1)
    gap = z - z.gather(1, y)
    # the target's own term stays out of the sums, so that nothing cancels
    others = torch.ones_like(z).scatter(1, y, 0.0)
    rest1, rest2 = (((gap / tau).exp() * others).sum(1) for tau in (1.0, 2.0))
    loss1, loss2 = rest1.log1p(), rest2.log1p()
    want = loss1 if op == "ce" else 0.5 * loss1 + 0.5 * 4.0 * loss2
    rel = 20 * (3 * 2.0 ** -24 + 1.6e-8 * dim / 16 + 2.0 ** -24) + 2.0 ** -22 + 64 * 2.0 ** -24 + 2.0 ** -22
    got = out["token_losses"][0].double()
    assert bool((got > 0).all())
    assert float((got / want - 1).abs().max()) <= rel
    assert abs(float(out["loss"][0]) / float(want.sum()) - 1) <= rel + 2.0 ** -23
    p1, p2 = gap.exp() * others / (1 + rest1).unsqueeze(1), (gap / 2).exp() * others / (1 + rest2).unsqueeze(1)
    p1 -= torch.zeros_like(p1).scatter(1, y, (rest1 / (1 + rest1)).unsqueeze(1))
    p2 -= torch.zeros_like(p2).scatter(1, y, (rest2 / (1 + rest2)).unsqueeze(1))
    dz = p1 if op == "ce" else 0.5 * p1 + 0.5 * 2.0 * p2
    got = out["gw"][0].double().t()[:tokens]
    # float32 products: three parts of a gradient, their sum scaled for one step of depth's cut at each k block
    rel += 2.0 ** -22 + (2 * 2.0 ** -11 + 2.0 ** -8 if dtype == BF16 else 2.0 ** -22 + 2.0 ** -18)
    assert float((got / dz - 1).abs().max()) <= rel


@pytest.mark.parametrize("tokens,vocab,dim", CONFIDENT)
@TYPES
@pytest.mark.parametrize("op", ["ce", "distill"])
@pytest.mark.parametrize("places", [[0, 1], [3, -1], [0, 50, 99], list(range(100))])
def test_equal_largest_logits_count_each(tokens, vocab, dim, dtype, op, places):
    # several columns hold the largest logit, in one unit of 128 and in many; the others lie 8 to 20 below
    x, z = _confident(tokens, vocab, dim, dtype, 64, seed=7)
    places = sorted({(p if p < 0 else p * vocab // 100) % vocab for p in places})
    w = x["weights"][0]
    w[:, :tokens] = torch.where(w[:, :tokens] == 64, torch.full_like(w[:, :tokens], 56), w[:, :tokens])
    w[places, :tokens] = 64
    x["targets"][0][:] = places[-1]
    x["indices"][0][:] = places[-1]
    z = w[:, :tokens].double().t()
    out = _run(x, op, grads=False, reduction=ddp.DDP_LOSS_SUM)
    loss1, loss2 = (-torch.log_softmax(z / tau, 1)[:, places[-1]] for tau in (1.0, 2.0))
    want = loss1 if op == "ce" else 0.5 * loss1 + 0.5 * 4.0 * loss2
    # as above, of losses from log 2 on; the sums' steps are relative to them, log 2 is 0.69
    rel = (20 * (4 * 2.0 ** -24 + 1.6e-8 * dim / 16) + 2 * 2.0 ** -22 + 64 * 2.0 ** -24) / 0.69
    assert float((out["token_losses"][0].double() / want - 1).abs().max()) <= rel


@pytest.mark.parametrize("tokens,vocab,dim", [(16, 100, 32), (300, 769, 128)])
@TYPES
@pytest.mark.parametrize("top", [15.0, 90.0, 1000.0])
def test_no_loss_is_below_zero(tokens, vocab, dim, dtype, top):
    # targets that lead by so much that nothing else counts; logits of no particular value
    gen = torch.Generator(device="cuda").manual_seed(5)
    kw = dict(device="cuda", generator=gen)
    x = _inputs([tokens], vocab, dim, dtype, seed=6)
    w = x["weights"][0].float()
    lean = top * (1.0 + torch.rand(tokens, 1, **kw)) / (w[x["targets"][0]] ** 2).sum(1, keepdim=True)
    x["hidden"][0] = (lean * w[x["targets"][0]]).to(dtype)
    for op in ("ce", "distill"):
        if op == "distill":
            x["indices"], x["teacher"] = [x["targets"][0].unsqueeze(1).contiguous()], [torch.zeros(tokens, 1, device="cuda")]
        out = _run(x, op)
        assert bool((out["token_losses"][0] >= 0).all()) and float(out["loss"][0]) >= 0
