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
