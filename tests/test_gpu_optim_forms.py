"""Kernel forms of AdamW and of the sync with norm that large models reach, against float64 and the sync without a norm.

AdamW takes two groups of four elements a thread above 4Mi elements over all ranks (but for fp32 gradients with copies),
and counts its steps in a launch of its own above 608 tiles; its tolerances are those of test_gpu_optim.

The sync goes element by element where the ranks' pointers lie differently against 16 bytes, and a block takes several
tiles under a CTA cap.  Norm tolerance there, with u = 2^-24: a thread adds at most 32 squares one behind the other (four
vectors of eight bf16; 16 of fp32), each square rounded once: 32 u; ten additions in the block: 42 u on the sum, 21 u on
its root; the sum's rounding to binary32 (half of it on the root) and the root's: 22.5 u.  23 u allowed.
"""
import math

import pytest
import torch

import gradient_sync_plan_gb300 as ddp
from gpu_util import guarded_copy
from test_gpu_optim import DT, U, _adamw64, _check_held, _moments, _norm64, _place, _values

pytestmark = pytest.mark.gpu

SPREAD = 4 << 20                       # elements from which on a thread takes two groups
LARGE = [1_500_003, 7, 600_001, 129, 40_000]
FORMS = [("f32", False), ("bf16", True), ("f32", True), ("bf16", False)]
HYPER = dict(lr=3e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1)


def _zeros(world, sizes):
    return [[torch.zeros(k) for k in sizes] for _ in range(world)]


def _check_step(new, old, factors, t, decays, ranks):
    """new, old: (p, m, v[, g]) as [r][i]; every element of `ranks` against float64."""
    h = HYPER
    for r in ranks:
        for i, decay in enumerate(decays):
            want = _adamw64(*[old[j][r][i] for j in range(4)], factors[r], t, h["lr"], h["b1"], h["b2"], h["eps"],
                            h["wd"] if decay else 0.0)
            for x, (y, tol), what in zip(new, want, "pmv"):
                d = (x[r][i].double() - y).abs()
                assert bool((d <= tol).all()), (what, r, i, float((d / tol).max()))


def _step(opt, norms, max_norm):
    h = HYPER
    opt.step(h["lr"], (h["b1"], h["b2"]), h["eps"], h["wd"], norms, max_norm)


@pytest.mark.parametrize("dtype,copies", FORMS)
@pytest.mark.parametrize("state,gradients", [("apart", "apart"), ("packed", "packed"), ("odd", "odd"), ("apart", "packed")])
@pytest.mark.parametrize("t0", [0, 1000])
def test_adamw_of_a_large_list(dtype, copies, state, gradients, t0):
    world = 2
    assert world * sum(LARGE) > SPREAD
    p, m, v = _moments(world, LARGE, 21, t0 == 0)
    (p, hp), (m, hm), (v, hv) = (_place(x, state, torch.float32) for x in (p, m, v))
    g, hg = _place(_values(world, LARGE, 30), gradients, DT[dtype])
    c, hc = _place(_zeros(world, LARGE), state, torch.bfloat16) if copies else (None, [])
    no_decay = [i % 3 == 1 for i in range(len(LARGE))]
    norms = torch.tensor([2.5, 0.25], device="cuda")
    opt = ddp.AdamW(p, g, m, v, copies=c, no_decay=no_decay,
                    steps=torch.full((world,), t0, dtype=torch.int32, device="cuda"))
    factors = [min(1.0, 1.0 / (float(n) + 1e-6)) for n in norms]
    for t in (t0 + 1, t0 + 2):
        old = [[[x.clone() for x in row] for row in k] for k in (p, m, v, g)]
        _step(opt, norms, 1.0)
        torch.cuda.synchronize()
        assert opt.steps.tolist() == [t] * world
        _check_step((p, m, v), old, factors, t, [not x for x in no_decay], range(world))
        assert all(torch.equal(a, b) for x, y in zip(g, old[3]) for a, b in zip(x, y)), "a gradient was written"
        if copies:
            assert all(torch.equal(a, b.bfloat16()) for x, y in zip(c, p) for a, b in zip(x, y))
    for held in (hp, hm, hv, hg, hc):
        _check_held(held, "adamw")


@pytest.mark.parametrize("dtype,copies,n", [(*f, 1_100_003) for f in FORMS] + [("bf16", False, 300_001), ("f32", False, 300_001)])
@pytest.mark.parametrize("cap", [0, 611])
def test_large_skipped_ranks_are_left_as_they_were(dtype, copies, n, cap):
    """The weights and the counts are two launches here, which have to agree on who is skipped."""
    world, sizes = 5, [n, 17]
    norms = torch.tensor([2.0, float("inf"), 0.5, float("nan"), 3e38], device="cuda")
    runs = [0, 2, 4]
    p, m, v = (_place(x, "apart", torch.float32)[0] for x in _moments(world, sizes, 3, False))
    g, _ = _place(_values(world, sizes, 9, 1.0), "apart", DT[dtype])
    c = _place(_values(world, sizes, 12, 1.0), "apart", torch.bfloat16)[0] if copies else None
    opt = ddp.AdamW(p, g, m, v, copies=c, steps=torch.tensor([4, 5, 4, 7, 4], dtype=torch.int32, device="cuda"))
    kinds = [p, m, v] + ([c] if copies else [])
    first = [[[x.clone() for x in row] for row in k] for k in kinds]
    factors = [min(1.0, 1.0 / (float(x) + 1e-6)) if math.isfinite(x) else 0.0 for x in norms.tolist()]
    previous = ddp.ddp_set_max_ctas(cap)
    try:
        for t in (5, 6):
            old = [[[x.clone() for x in row] for row in k] for k in (p, m, v, g)]
            _step(opt, norms, 1.0)
            torch.cuda.synchronize()
            assert opt.steps.tolist() == [t, 5, t, 7, t]
            _check_step((p, m, v), old, factors, t, [True, True], runs)
            if copies:
                assert all(torch.equal(c[r][i], p[r][i].bfloat16()) for r in runs for i in range(2))
            for k, before in zip(kinds, first):
                assert all(torch.equal(k[r][i], before[r][i]) for r in (1, 3) for i in range(2)), "a skipped rank was written"
    finally:
        ddp.ddp_set_max_ctas(previous)


# --------------------------------------------------------------------------
# The sync that returns the norm
# --------------------------------------------------------------------------

def _place_shifted(rows, dtype):
    """_place with rank r's tensors r elements past an aligned address."""
    out, held = [], []
    step = 512 // (2 if dtype == torch.bfloat16 else 4)
    for r, row in enumerate(rows):
        offs, at = [], 0
        for t in row:
            offs.append(at + r % 8)
            at = -(-(offs[-1] + t.numel()) // step) * step
        storage, flat = guarded_copy(torch.zeros(at, dtype=dtype))
        views = [flat[o:o + t.numel()] for o, t in zip(offs, row)]
        for v, t in zip(views, row):
            v.copy_(t.to(dtype))
        gaps = torch.ones(flat.numel(), dtype=torch.bool)
        for o, t in zip(offs, row):
            gaps[o:o + t.numel()] = False
        held.append((storage, flat, gaps.cuda()))
        out.append(views)
    return out, held


def _algos(dtype):
    return [ddp.DDP_ALGO_VIEW] + ([] if dtype == "bf16" else [ddp.DDP_ALGO_BF16_HOOK_VIEW, ddp.DDP_ALGO_FP16_HOOK_VIEW])


def _equal(a, b):
    return all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


def _check_norms(norms, row, world):
    want = _norm64(row)
    assert norms.shape == (world,) and bool((norms == norms[0]).all())
    assert abs(float(norms[0]) - want) <= 23 * U * want


@pytest.mark.parametrize("dtype,algo", [(d, a) for d in ("f32", "bf16") for a in _algos(d)])
@pytest.mark.parametrize("world,sizes", [
    (2, [5_100_003, 33, 900]), (3, [5_100_003, 33, 900]), (3, [10_000_019]), (5, [700, 3, 257, 1]), (8, [1_000_003, 5, 40_001]),
    (9, [2048, 30]), (20, [50_001, 300]),
])
def test_sync_norm_over_ranks_of_unlike_alignment(world, sizes, dtype, algo):
    rows = _values(world, sizes, 8, 1e-2)
    views, held = _place_shifted(rows, DT[dtype])
    other, _ = _place_shifted(rows, DT[dtype])
    plan = ddp.ddp_plan_buckets(sizes, ddp.BF16 if dtype == "bf16" else ddp.F32, 64 << 10, 1 << 20)
    ddp.ddp_sync_buckets(other, plan, None, algo=algo)
    norms = ddp.SyncNormCall(views, plan, algo=algo)()
    torch.cuda.synchronize()
    _check_held(held, "sync norm")
    assert _equal(views, other)
    _check_norms(norms, views[0], world)


@pytest.mark.parametrize("shifted", [False, True], ids=["aligned", "shifted"])
@pytest.mark.parametrize("extreme", [False, True], ids=["usual", "extreme"])
@pytest.mark.parametrize("dtype,algo", [("f32", ddp.DDP_ALGO_VIEW), ("bf16", ddp.DDP_ALGO_VIEW),
                                        ("f32", ddp.DDP_ALGO_BF16_HOOK_VIEW)])
@pytest.mark.parametrize("world,sizes", [(2, [7_000_001, 77]), (4, [7_000_001, 77]), (8, [6_000_001, 77, 100_003])])
def test_sync_norm_with_several_tiles_a_block(world, sizes, dtype, algo, extreme, shifted):
    """A cap that leaves the register kernel on but has fewer CTAs than there are tiles; some tiles' squares leave
    binary32's range (two parts of the largest tensor, beside usual and zero ones) and are taken again."""
    rows = _values(world, sizes, 5, 1e-2)
    if extreme:
        for row in rows:
            row[0][100_000:900_000] *= 1e-25
            row[0][2_000_000:2_100_000] = 0.0
            row[0][3_000_000:3_700_000] *= 1e24
    place = _place_shifted if shifted else lambda r, d: _place(r, "apart", d)
    (views, held), (other, _), (free, _) = (place(rows, DT[dtype]) for _ in range(3))
    plan = ddp.ddp_plan_buckets(sizes, ddp.BF16 if dtype == "bf16" else ddp.F32)
    ddp.ddp_sync_buckets(other, plan, None, algo=algo)
    want = ddp.SyncNormCall(free, plan, algo=algo)().clone()
    cap = 4 * torch.cuda.get_device_properties(0).multi_processor_count + 1
    previous = ddp.ddp_set_max_ctas(cap)
    try:
        norms = ddp.SyncNormCall(views, plan, algo=algo)()
        torch.cuda.synchronize()
    finally:
        ddp.ddp_set_max_ctas(previous)
    _check_held(held, "sync norm")
    assert _equal(views, other) and _equal(free, other)
    assert torch.equal(norms, want), "the cap changed the norm"
    _check_norms(norms, views[0], world)
