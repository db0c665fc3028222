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
         ([300], 1000, 256), ([257, 300], 391, 515), ([40], 5003, 7), ([33], 127, 1000), ([1], 20000, 3), ([2, 1], 1030, 64),
         ([3], 1, 20000), ([0, 5], 700, 40), ([256], 256, 256), ([512, 1024], 129, 72), ([250], 3000, 520), ([2500], 4500, 24),
         ([4200], 300, 21)]


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
                                                       (0.5, 1.0, True), (0.4, 0.5, True), (9.0, 0.5, True)])
@pytest.mark.parametrize("tokens,vocab,dim,k", [([5], 40, 32, 1), ([16, 7], 100, 32, 8), ([130, 200], 777, 128, 64), ([500, 512], 515, 72, 20),
                                                ([64], 300, 66, 256), ([3, 1], 1100, 64, 5)])
def test_distillation(tokens, vocab, dim, k, temperature, alpha, targets, dtype):
    x = _inputs(tokens, vocab, dim, dtype, ignored=0.2 if targets else 0.0, seed=k + dim, teacher=k)
    how = dict(temperature=temperature, alpha=alpha, targets=targets)
    run = Run(x)
    run.check(run.distill(reduction="mean", **how), distill=True, reduction="mean", **how)
    alone = Run(x, grads=False)
    alone.check(alone.distill(grad=False, reduction="world_mean", **how), grad=False, distill=True, reduction="world_mean", **how)


SMALL, TILES = ([16, 7], 100, 32), ([130, 40], 777, 128)      # one launch; the tensor cores' kernels
PAIRS = ([512, 500], 777, 200)                                # whose blocks work in pairs
BOTH = pytest.mark.parametrize("tokens,vocab,dim", [SMALL, TILES, PAIRS])
TYPES = pytest.mark.parametrize("dtype", [BF16, F32])


@BOTH
@TYPES
def test_nothing_of_an_ignored_token_is_read(tokens, vocab, dim, dtype):
    x = _inputs(tokens, vocab, dim, dtype, ignored=0.4, seed=3, teacher=8)
    for r in range(len(tokens)):
        skip = x["targets"][r] == IGNORE
        assert bool(skip.any())
        x["hidden"][r][skip] = float("nan")
        x["teacher"][r][skip] = float("inf")
    run = Run(x)
    run.check(run.ce())
    assert all(bool((g[t == IGNORE] == 0).all()) for g, t in zip(run.gh, x["targets"]))
    run = Run(x)
    run.check(run.distill(alpha=0.5, temperature=2.0), distill=True, alpha=0.5, temperature=2.0)


@BOTH
@TYPES
@pytest.mark.parametrize("reduction", ["sum", "mean", "world_mean"])
def test_a_rank_without_learned_tokens(tokens, vocab, dim, dtype, reduction):
    x = _inputs(tokens, vocab, dim, dtype, seed=4)
    x["targets"][0][:] = IGNORE
    run = Run(x)
    loss = run.ce(reduction=reduction)
    run.check(loss, reduction=reduction)
    assert float(loss[0]) == 0.0 and bool((run.gw[0] == 0).all()) and bool((run.gh[0] == 0).all())
    x["targets"][1][:] = IGNORE
    loss = run.ce(reduction=reduction)
    torch.cuda.synchronize()
    assert loss.tolist() == [0.0, 0.0] and all(bool((g == 0).all()) for g in run.gw + run.gh)


@BOTH
@TYPES
def test_teachers_with_padding_duplicates_and_lowest_logits(tokens, vocab, dim, dtype):
    x = _inputs(tokens, vocab, dim, dtype, seed=5, teacher=12, ignored=0.1)
    low = torch.finfo(F32).min
    for r in range(len(tokens)):
        i, t = x["indices"][r], x["teacher"][r]
        i[0, 3:] = -1                                     # fewer entries
        t[1, 5:] = -float("inf")
        i[2, 1::2] = i[2, 0]                              # one column often
        i[3, :] = i[3, 0]                                 # and always
        t[4, 1:] = low                                    # masked by the lowest value
        t[5, :] = low
        i[6, :] = -1                                      # none at all
        i[:, 7] = torch.where(x["targets"][r] >= 0, x["targets"][r], i[:, 7])       # the target among them, and once more
        i[6, :] = -1
    for how in (dict(alpha=1.0, temperature=1.0, targets=False), dict(alpha=0.4, temperature=2.0, targets=True),
                dict(alpha=1.0, temperature=0.5, targets=True)):
        run = Run(x)
        run.check(run.distill(**how), distill=True, **how)
        assert float(run.losses[0][6]) == 0.0


@BOTH
def test_bf16_teachers(tokens, vocab, dim):
    x = _inputs(tokens, vocab, dim, seed=6, teacher=9)
    x["teacher"] = [t.bfloat16() for t in x["teacher"]]
    run = Run(x)
    run.check(run.distill(alpha=0.5, temperature=2.0), distill=True, alpha=0.5, temperature=2.0)


@BOTH
@TYPES
def test_columns_outside_the_vocabulary_are_reported_and_left_out(tokens, vocab, dim, dtype):
    for bad in (vocab, -7, 1 << 40):
        x = _inputs(tokens, vocab, dim, dtype, seed=7, teacher=4)
        x["targets"][1][2] = bad
        run = Run(x)
        loss = run.ce()
        torch.cuda.synchronize()
        assert ddp.ddp_device_status() == -1 and ddp.ddp_device_status() == 0       # DDP_ERR_INVALID, then cleared
        run.check(loss)
    x = _inputs(tokens, vocab, dim, dtype, seed=8, teacher=4)
    x["indices"][0][1, 2] = vocab
    run = Run(x)
    loss = run.distill(targets=False)
    torch.cuda.synchronize()
    assert ddp.ddp_device_status() == -1
    run.check(loss, distill=True, targets=False)


@BOTH
@TYPES
def test_an_ignored_value_that_is_a_column(tokens, vocab, dim, dtype):
    x = _inputs(tokens, vocab, dim, dtype, seed=9)
    x["targets"][0][:4] = 5
    run = Run(x)
    run.check(run.ce(ignore_index=5), ignore=5)


@BOTH
@TYPES
def test_accumulation_adds_with_one_rounding(tokens, vocab, dim, dtype):
    x = _inputs(tokens, vocab, dim, dtype, seed=10, ignored=0.2)
    first = Run(x)
    first.ce(scale=2.0)
    run = Run(x)
    old = [torch.randn(vocab, dim, device="cuda").to(dtype) * 1e-2 for _ in tokens]
    for g, o in zip(run.gw, old):
        g.copy_(o)
    loss = run.ce(scale=2.0, accumulate=True)
    torch.cuda.synchronize()
    want = loss_ref.reference(x["hidden"], x["weights"], x["targets"], scale=2.0)
    for r, w in enumerate(want):
        # the gradient's bound has a rounding of its own, the sum one more
        total = old[r].double() + w["grad_weights"]
        bound = w["weights_bound"] + total.abs() * loss_ref.half_step(dtype)
        assert bool(((run.gw[r].double() - total).abs() <= bound).all())
        assert torch.equal(run.gh[r], first.gh[r])
    x["targets"][0][:] = IGNORE                           # nothing learned: nothing added
    run.gw[0].copy_(old[0])
    run.ce(accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(run.gw[0], old[0])


@BOTH
@TYPES
def test_hidden_states_in_wider_rows(tokens, vocab, dim, dtype):
    x = _inputs(tokens, vocab, dim, dtype, seed=11)
    plain = Run(x)
    plain.ce()
    for pad in (1, 8, 24):
        wide = [torch.full((n, dim + pad), float("nan"), dtype=dtype, device="cuda") for n in tokens]
        for start in {0, pad}:
            views = [v[:, start:start + dim] for v in wide]
            for v, h in zip(views, x["hidden"]):
                v.copy_(h)
            run = Run(dict(x, hidden=views))
            run.gh = [torch.full((n, dim), float("nan"), dtype=dtype, device="cuda") for n in tokens]
            run.ce()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(run.gh + run.gw + run.losses, plain.gh + plain.gw + plain.losses))


@TYPES
@pytest.mark.parametrize("dim", [32, 33, 130, 128])
def test_tensors_at_odd_addresses(dtype, dim):
    tokens, vocab = [70], 601
    x = _inputs(tokens, vocab, dim, dtype, seed=12)
    plain = Run(x)
    plain.ce()

    def moved(t, by):
        flat = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
        return flat[by:].view(t.shape)

    run = Run(x)
    run.gw = [moved(run.gw[0], 1)]
    weights = x["weights"]
    if dtype == F32 or dim % 64:                          # other bf16 weights start on 16-byte boundaries
        weights = [moved(weights[0], 1).copy_(weights[0])]
    run.head = ddp.LossHead(weights, run.gw, max_tokens=70)
    x["hidden"] = [moved(x["hidden"][0], 3).copy_(x["hidden"][0])]
    run.gh = [moved(run.gh[0], 1)]
    run.losses = [moved(run.losses[0], 1)]
    run.ce()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(run.gh + run.gw + run.losses, plain.gh + plain.gw + plain.losses))


@BOTH
def test_repeats_caps_and_larger_handles_change_nothing(tokens, vocab, dim):
    x = _inputs(tokens, vocab, dim, seed=13, teacher=6, ignored=0.2)
    runs = [Run(x), Run(x, max_teacher=40), Run(x), Run(x)]
    for run, cap in zip(runs, (0, 0, 3, 1)):
        previous = ddp.ddp_set_max_ctas(cap)
        try:
            for _ in range(2):
                run.distill(alpha=0.5, temperature=2.0, reduction="world_mean")
        finally:
            ddp.ddp_set_max_ctas(previous)
    torch.cuda.synchronize()
    for run in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(run.gh + run.gw + run.losses, runs[0].gh + runs[0].gw + runs[0].losses))


@pytest.mark.parametrize("world,tokens,vocab,dim", [(18, 5, 90, 24), (17, 9, 300, 72)])
@pytest.mark.parametrize("distill", [False, True])
def test_more_ranks_than_a_launch_takes(world, tokens, vocab, dim, distill):
    x = _inputs([tokens] * world, vocab, dim, seed=14, ignored=0.3, teacher=4)
    run = Run(x)
    if distill:
        run.check(run.distill(reduction="world_mean", alpha=0.5), distill=True, alpha=0.5, reduction="world_mean")
    else:
        run.check(run.ce(reduction="world_mean"), reduction="world_mean")


@BOTH
def test_a_captured_call_replays_on_new_values(tokens, vocab, dim):
    x = _inputs(tokens, vocab, dim, seed=15, teacher=6, ignored=0.2)
    run = Run(x)
    run.distill(alpha=0.5, temperature=2.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = run.distill(alpha=0.5, temperature=2.0)
    other = _inputs(tokens, vocab, dim, seed=16, teacher=6, ignored=0.4)
    for k in ("hidden", "targets", "teacher", "indices", "weights"):
        for a, b in zip(x[k], other[k]):
            a.copy_(b)
    graph.replay()
    run.check(loss, distill=True, alpha=0.5, temperature=2.0)


@BOTH
def test_another_stream_and_another_output(tokens, vocab, dim):
    x = _inputs(tokens, vocab, dim, seed=17)
    run = Run(x)
    out = torch.empty(len(tokens), device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    assert run.ce(stream=stream, out=out) is out
    stream.synchronize()
    run.check(out)


def test_extreme_logits():
    # a weight row that every hidden state sees at +-1e4, far beyond what exp takes
    x = _inputs([40], 700, 64, seed=18)
    x["weights"][0][5] = 0
    x["weights"][0][5, 0] = 1e4
    x["hidden"][0][:, 0] = torch.where(torch.arange(40, device="cuda") % 2 == 0, 1.0, -1.0).to(BF16)
    x["targets"][0][::4] = 5
    run = Run(x)
    loss = run.ce()
    torch.cuda.synchronize()
    want = loss_ref.reference(x["hidden"], x["weights"], x["targets"])
    loss_ref.check(want, loss, run.losses, run.gh, run.gw)


@TYPES
def test_pieces_of_the_vocabulary(dtype):
    # more logits than the workspace keeps: 16-bit exponentials of 8320 x 131200 take 2.03 GiB, so the vocabulary goes in pieces
    tokens, vocab, dim = [8320 if dtype == BF16 else 2000], 131200, 8
    x = _inputs(tokens, vocab, dim, dtype, seed=19, ignored=0.1)
    run = Run(x)
    loss = run.ce()
    torch.cuda.synchronize()
    # against the same in float32, token by token in parts (float64 of all logits would be 8.7 GB)
    keep = x["targets"][0] != IGNORE
    h, w, y = x["hidden"][0][keep].double(), x["weights"][0].double(), x["targets"][0][keep]
    n = h.shape[0]
    gh, gw, losses = torch.zeros_like(h), torch.zeros_like(w), torch.zeros(n, dtype=torch.float64, device="cuda")
    for a in range(0, n, 1024):
        z = h[a:a + 1024] @ w.t()
        logp = torch.log_softmax(z, 1)
        k = y[a:a + 1024].unsqueeze(1)
        losses[a:a + 1024] = -logp.gather(1, k).squeeze(1)
        dz = logp.exp()
        dz.scatter_add_(1, k, -torch.ones_like(k, dtype=torch.float64))
        dz /= n
        gh[a:a + 1024] = dz @ w
        gw += dz.t() @ h[a:a + 1024]
    off = lambda got, want: float((got.double() - want).norm() / want.norm())
    # norms: a rounding of the logits' gradients and one of the result, each below a half step; three-part sums 2^-18
    most = 2 * loss_ref.half_step(dtype) if dtype == BF16 else 2.0 ** -16
    assert abs(float(loss[0]) / float(losses.mean()) - 1) < 2.0 ** -18
    assert off(run.losses[0][keep], losses) < 2.0 ** -18
    assert off(run.gh[0][keep], gh) < most and off(run.gw[0], gw) < most
    assert ddp.ddp_device_status() == 0
