"""Refusals of the loss head's entry points, and its workspace's size.

Every call here is refused by the host checks or makes a head, which makes no CUDA call, so no made-up pointer reaches
the GPU.
"""
import ctypes
import math

import pytest
import torch

import gradient_sync_plan_gb300 as ddp
import loss_ref

H = 0x7f0000000000                     # made-up device addresses, never dereferenced
STEP = 1 << 32
WS = H + (1 << 44)
LOSS = H + (1 << 45)
INF, NAN = float("inf"), float("nan")


def _vp(*p):
    return (ctypes.c_void_p * max(len(p), 1))(*p)


def _i32(*v):
    return (ctypes.c_int32 * max(len(v), 1))(*v)


def _bytes(world=2, vocab=100, dim=32, dtype=1, max_tokens=16, max_teacher=8, grads=1, out=True):
    n = ctypes.c_int64(-1)
    st = ddp.lib().ddp_loss_head_workspace_bytes(world, vocab, dim, dtype, max_tokens, max_teacher, grads,
                                                 ctypes.byref(n) if out else None)
    return st, n.value


def _create(world=2, weights=None, grads=None, vocab=100, dim=32, dtype=1, max_tokens=16, max_teacher=8, ws=WS, ws_bytes=None,
            out=True):
    weights = [H + r * STEP for r in range(world)] if weights is None else weights
    grads = [H + (world + r) * STEP for r in range(world)] if grads is None else grads
    h = ctypes.c_void_p(1)
    n = 1 << 50 if ws_bytes is None else ws_bytes
    if ws_bytes is None:
        st, n = _bytes(world, vocab, dim, dtype, max_tokens, max_teacher, 1 if grads else 0)
        n = n if st == 0 else 1 << 40
    st = ddp.lib().ddp_loss_head_create(world, _vp(*weights) if weights != [] else None, _vp(*grads) if grads else None, vocab, dim,
                                        dtype, max_tokens, max_teacher, ws, n, ctypes.byref(h) if out else None)
    assert not out or st == 0 or h.value is None
    return st, h


@pytest.mark.parametrize("want,kw", [
    (-1, dict(world=0)), (-5, dict(world=513)), (-1, dict(dtype=2)), (-1, dict(vocab=0)), (-1, dict(dim=0)), (-1, dict(max_tokens=0)),
    (-1, dict(max_teacher=-1)), (-5, dict(vocab=ddp.DDP_MAX_VOCAB + 1)), (-5, dict(dim=ddp.DDP_MAX_DIM + 1)),
    (-5, dict(max_teacher=ddp.DDP_MAX_TEACHER + 1)), (-5, dict(max_tokens=(1 << 28) // 2 + 1)),
    (-5, dict(world=1, vocab=1 << 24, max_tokens=1 << 22)), (-1, dict(out=False)),
])
def test_sizes_that_are_refused(want, kw):
    assert _bytes(**kw)[0] == want
    if kw.get("max_tokens", 0) == 0:
        assert _create(**kw)[0] == want


@pytest.mark.parametrize("want,kw", [
    (-1, dict(weights=[])), (-1, dict(weights=[H, None])), (-1, dict(ws=None)), (-2, dict(ws=WS + 16)), (-5, dict(ws_bytes=100)),
    (-1, dict(grads=[H + STEP, None])), (-2, dict(grads=[H + 2 * STEP + 1, H + 3 * STEP])), (-2, dict(weights=[H + 1, H + STEP])),
    (-1, dict(grads=[H + 2 * STEP, H + 2 * STEP + 6398])),        # the second begins in the first's last element
    (-1, dict(grads=[H, H + 3 * STEP])),                          # in the weights
    (-1, dict(ws=H + 3 * STEP)),                                  # the workspace over the second rank's gradients
    (-2, dict(weights=[H + 8, H + STEP], dim=64)),                # bf16 rows of whole boxes are read where they are
    (-2, dict(weights=[H + 2, H + STEP], dtype=0)),
])
def test_tensors_that_are_refused(want, kw):
    assert _create(**kw)[0] == want


def test_heads_that_are_taken():
    for kw in (dict(), dict(grads=[]), dict(weights=[H + 2, H + STEP]), dict(dtype=0, weights=[H + 4, H + STEP]),
               dict(weights=[H, H]), dict(world=17), dict(max_teacher=0)):
        st, h = _create(**kw)
        assert st == 0
        assert ddp.lib().ddp_loss_head_destroy(h) == 0
    assert ddp.lib().ddp_loss_head_destroy(None) == 0


def _args(world=2, **kw):
    at = lambda k: [H + (40 + 4 * k + r) * STEP for r in range(world)]
    args = dict(tokens=[16, 7], hidden=at(0), stride=32, teacher_n=8, teacher=at(1), teacher_dtype=0, indices=at(2), temperature=2.0,
                alpha=0.5, targets=at(3), ignore=-100, reduction=1, scale=1.0, accumulate=0, token_losses=at(4), loss=LOSS,
                grad_hidden=at(5))
    args.update(kw)
    return args


def _table(p):
    return None if p is None else _vp(*p)


def _call(h, fn, a):
    tokens = None if a["tokens"] is None else _i32(*a["tokens"])
    args = [h, tokens, _table(a["hidden"]), a["stride"]]
    if "distill" in fn:
        args += [a["teacher_n"], _table(a["teacher"]), a["teacher_dtype"], _table(a["indices"]), a["temperature"], a["alpha"]]
    args += [_table(a["targets"]), a["ignore"], a["reduction"]]
    if fn.endswith("grad"):
        args += [a["scale"], a["accumulate"]]
    args += [_table(a["token_losses"]), a["loss"]]
    if fn.endswith("grad"):
        args.append(_table(a["grad_hidden"]))
    return getattr(ddp.lib(), fn)(*args, None)


FNS = ["ddp_cross_entropy", "ddp_cross_entropy_grad", "ddp_distill", "ddp_distill_grad"]
X = H + 60 * STEP


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("want,kw", [
    (-1, dict(tokens=None)), (-1, dict(tokens=[16, -1])), (-5, dict(tokens=[17, 1])), (-1, dict(hidden=None)),
    (-1, dict(hidden=[X, None])), (-2, dict(hidden=[X + 1, X + STEP])), (-1, dict(stride=31)), (-5, dict(stride=1 << 62)),
    (-1, dict(reduction=-1)), (-1, dict(reduction=3)), (-1, dict(loss=None)), (-2, dict(loss=LOSS + 2)), (-1, dict(loss=WS + 64)),
    (-1, dict(loss=H + 4)),                                       # in the weights
    (-2, dict(targets=[X + 4, X + STEP])), (-1, dict(targets=[X, None])), (-2, dict(token_losses=[X + 2, X + STEP])),
    (-1, dict(token_losses=[X, X + 60])),                         # the second begins in the first's last element
    (-1, dict(token_losses=[LOSS + 4, X])),                       # over the second rank's loss
])
def test_calls_that_are_refused(fn, want, kw):
    st, h = _create()
    assert st == 0
    assert _call(h, fn, _args(**kw)) == want
    assert _call(None, fn, _args()) == -1
    ddp.lib().ddp_loss_head_destroy(h)


@pytest.mark.parametrize("fn", ["ddp_distill", "ddp_distill_grad"])
@pytest.mark.parametrize("want,kw", [
    (-1, dict(teacher_n=0)), (-5, dict(teacher_n=9)), (-1, dict(teacher=None)), (-1, dict(indices=None)), (-1, dict(teacher_dtype=2)),
    (-2, dict(teacher=[X + 2, X + STEP])), (-2, dict(indices=[X + 4, X + STEP])), (-1, dict(indices=[None, X])),
    (-1, dict(temperature=0.0)), (-1, dict(temperature=-1.0)), (-1, dict(temperature=NAN)), (-1, dict(temperature=INF)),
    (-1, dict(temperature=1e-60)), (-1, dict(temperature=1e-39)), (-1, dict(alpha=0.0)), (-1, dict(alpha=1.5)), (-1, dict(alpha=NAN)),
    (-1, dict(alpha=-0.5)), (-1, dict(alpha=1e-60)), (-1, dict(targets=None)),     # alpha 0.5 needs targets
])
def test_distillations_that_are_refused(fn, want, kw):
    st, h = _create()
    assert st == 0
    assert _call(h, fn, _args(**kw)) == want
    ddp.lib().ddp_loss_head_destroy(h)


@pytest.mark.parametrize("fn", ["ddp_cross_entropy_grad", "ddp_distill_grad"])
@pytest.mark.parametrize("want,kw", [
    (-1, dict(scale=INF)), (-1, dict(scale=NAN)), (-1, dict(scale=1e60)), (-1, dict(grad_hidden=None)),
    (-1, dict(grad_hidden=[X, None])), (-2, dict(grad_hidden=[X + 1, X + STEP])),
    (-1, dict(grad_hidden=[X, X + 1022])),                        # rank 0's 16 x 32 bf16 end two bytes later
    (-1, dict(grad_hidden=[H + 40 * STEP, X])),                   # in place of the hidden states
])
def test_gradients_that_are_refused(fn, want, kw):
    st, h = _create()
    assert st == 0
    assert _call(h, fn, _args(**kw)) == want
    ddp.lib().ddp_loss_head_destroy(h)
    st, h = _create(grads=[])
    assert st == 0 and _call(h, fn, _args()) == -1               # a head without gradients
    ddp.lib().ddp_loss_head_destroy(h)


def test_targets_are_needed_for_cross_entropy():
    st, h = _create()
    assert st == 0
    assert _call(h, "ddp_cross_entropy", _args(targets=None)) == -1
    assert _call(h, "ddp_cross_entropy_grad", _args(targets=None)) == -1
    ddp.lib().ddp_loss_head_destroy(h)


def test_workspace_grows_with_what_it_holds_and_is_bounded():
    need = lambda **kw: _bytes(**kw)[1]
    assert need() > need(grads=0) > 0 and need(max_teacher=0) < need() and need(max_tokens=4000) > need()
    # 16-bit exponentials are kept up to 2 GiB, beyond that the vocabulary goes in pieces
    small, large = (need(world=1, vocab=131072, dim=64, max_tokens=n, max_teacher=0) for n in (8192, 65536))
    assert small > 2 << 30
    logits = 65536 * 131072 * 2
    assert large < logits / 2


def test_python_refusals():
    cpu = torch.zeros(100, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ddp.LossHead([cpu], max_tokens=4)                         # host memory
    with pytest.raises((ValueError, TypeError)):
        ddp.LossHead([cpu.half()], max_tokens=4)
    with pytest.raises((ValueError, ddp.DDPError, IndexError)):
        ddp.LossHead([], max_tokens=4)


def test_reference_against_torch_and_differences():
    """The tests' own reference: torch's losses, autograd, and differences of the loss."""
    gen = torch.Generator().manual_seed(0)
    w = torch.randn(13, 6, generator=gen, dtype=torch.float32).double()
    h = torch.randn(5, 6, generator=gen, dtype=torch.float32).double()
    y = torch.tensor([3, -100, 12, 0, 7])
    t = torch.randn(5, 4, generator=gen)
    i = torch.stack([torch.randperm(13, generator=gen)[:4] for _ in range(5)])

    def soft(hh, ww, a, tau):
        z = hh @ ww.t()
        q = torch.softmax(t.double() / tau, 1)
        logp = torch.log_softmax(z / tau, 1).gather(1, i)
        kl = torch.nn.functional.kl_div(logp, q, reduction="none").sum(1)
        ce = torch.nn.functional.cross_entropy(z, y, reduction="none")
        keep = (y != -100).double()
        return ((a * tau * tau * kl + (1 - a) * ce) * keep).sum() / keep.sum()

    x = loss_ref.reference([h.float()], [w.float()], [y], reduction="mean")[0]
    assert math.isclose(x["loss"], float(torch.nn.functional.cross_entropy(h @ w.t(), y)), rel_tol=1e-12)
    for a, tau in ((0.5, 2.0), (1.0, 1.0), (0.25, 0.5)):
        x = loss_ref.reference([h.float()], [w.float()], [y], [t], [i], temperature=tau, alpha=a, reduction="mean")[0]
        hh, ww = h.clone().requires_grad_(), w.clone().requires_grad_()
        loss = soft(hh, ww, a, tau)
        loss.backward()
        assert math.isclose(x["loss"], float(loss.detach()), rel_tol=1e-12)
        assert torch.allclose(x["grad_hidden"], hh.grad, rtol=1e-11, atol=1e-13)
        assert torch.allclose(x["grad_weights"], ww.grad, rtol=1e-11, atol=1e-13)
        # differences: error of second order in the step, 1e-5, and 2^-52 / 1e-5 of rounding
        for k in ((0, 0), (2, 5), (4, 3)):
            d = torch.zeros_like(h)
            d[k] = 1e-5
            slope = (soft(h + d, w, a, tau) - soft(h - d, w, a, tau)) / 2e-5
            assert abs(float(slope - x["grad_hidden"][k])) < 1e-8
