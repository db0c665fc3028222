"""Gradient norm, clipping, norm-in-sync and AdamW on the GPU against float64.

Tolerances, from the roundings on the way (u = 2^-24, binary32's unit roundoff):
  norm    positive terms, added as a tree: a thread's chains of at most 12
          squares (16 of scaled ones, where squares leave binary32's range), 3
          additions of its own and 10 in the block: below 30 u on the sum, half
          on its root, one rounding to binary32.  16 u allowed.
  clip    c: one add, one quotient; the product: 3 u, and the constant 1e-6's
          own rounding; 4 u allowed, for bf16 one rounding of 2^-8 on top.
  AdamW   m: 6 u of the sum of its two terms' sizes (they may cancel); v: 16 u
          (positive terms, g' squared carries 3 u twice); p: 2 u of p, 32 u of
          the update, and m's own error through it.
"""
import math

import numpy as np
import pytest
import torch

import gradient_sync_plan_gb300 as ddp
import workloads
from gpu_util import assert_canaries, guarded_copy

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -149
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _place(rows, layout, dtype):
    """Device tensors rows[r][i] (float64 CPU values rounded to dtype), as views: 'apart' (512-byte aligned), 'packed'
    (back to back from an aligned start) or 'odd' (each one element past an aligned start)."""
    out, held = [], []
    for row in rows:
        step = max(512 // (2 if dtype == torch.bfloat16 else 4), 1)
        offs, at = [], 0
        for t in row:
            offs.append(at + (1 if layout == "odd" else 0))
            at = offs[-1] + t.numel()
            if layout != "packed":
                at = -(-at // step) * step
        storage, flat = guarded_copy(torch.zeros(max(at, 1), dtype=dtype))
        views = [flat[o:o + t.numel()] for o, t in zip(offs, row)]
        for v, t in zip(views, row):
            v.copy_(t.to(dtype))
        gaps = torch.ones(flat.numel(), dtype=torch.bool)
        for o, t in zip(offs, row):
            gaps[o:o + t.numel()] = False
        held.append((storage, flat, gaps.cuda()))
        out.append(views)
    return out, held


def _check_held(held, what):
    for storage, flat, gaps in held:
        assert_canaries(storage, what)
        assert not bool(flat[gaps].any()), f"{what}: written between the tensors"


def _values(world, sizes, seed, scale=None):
    g = torch.Generator().manual_seed(seed)
    return [[torch.randn(n, generator=g, dtype=torch.float64) * (scale if scale else 10.0 ** (i % 5 - 3))
             for i, n in enumerate(sizes)] for _ in range(world)]


def _norm64(row):
    return math.sqrt(math.fsum(float(t.double().pow(2).sum()) for t in row))


SIZES = {
    "one": [1],
    "empty": [0, 0],
    "some_empty": [0, 5, 0, 1],
    "edges": [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 33, 127, 129],
    "tile": [4096, 4095, 4097, 8192, 8191, 8193, 1],
    "mixed": [100003, 7, 65536, 12345, 1, 300],
    "many": [1 + (37 * i) % 211 for i in range(1401)],
    "large": [5_000_011, 64, 2_000_000],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["apart", "packed", "odd"])
@pytest.mark.parametrize("sizes", SIZES, ids=list(SIZES))
@pytest.mark.parametrize("world", [1, 3])
def test_norm_and_clip(world, sizes, layout, dtype):
    rows = _values(world, SIZES[sizes], 7)
    views, held = _place(rows, layout, DT[dtype])
    before = [[v.clone() for v in row] for row in views]
    want = [_norm64(row) for row in before]
    s = ddp.GradSet(views)
    norms = s.norm()
    torch.cuda.synchronize()
    _check_held(held, "norm")
    for r in range(world):
        assert abs(float(norms[r]) - want[r]) <= 16 * U * want[r]
        assert all(torch.equal(a, b) for a, b in zip(views[r], before[r])), "norm wrote a gradient"
    first = norms.clone()
    assert torch.equal(s.norm().clone(), first), "a repeat changed a bit"
    limit = [1e-3, 0.7 * max(want) + 1e-9][world > 1]            # every rank, or only some, above it
    got = s.norm_clip(limit)
    torch.cuda.synchronize()
    assert torch.equal(got, first)
    _check_held(held, "clip")
    for r in range(world):
        c = min(1.0, limit / (float(first[r]) + 1e-6))
        for a, b in zip(views[r], before[r]):
            if c == 1.0:
                assert torch.equal(a, b)
                continue
            y = b.double() * c
            tol = (4 * U + (2.0 ** -8 if dtype == "bf16" else 0.0)) * y.abs() + (2.0 ** -133 if dtype == "bf16" else TINY)
            assert bool(((a.double() - y).abs() <= tol).all())
    s.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-23, 1e-19, 1e15, 3e18, 1e20, 1e30])
@pytest.mark.parametrize("n", [1, 1000, 300_001])
def test_norm_beyond_the_range_of_binary32_squares(n, scale, dtype):
    rows = _values(1, [n, 3], 3, scale)
    views, _ = _place(rows, "apart", DT[dtype])
    want = _norm64(views[0])
    got = float(ddp.GradSet(views).norm()[0])
    assert abs(got - want) <= 16 * U * want + TINY


def test_norm_of_huge_and_tiny_tensors_together():
    rows = [[torch.full((5000,), 1e-30, dtype=torch.float64), torch.full((5000,), 2e25, dtype=torch.float64),
             torch.full((70000,), 1.0, dtype=torch.float64)]]
    views, _ = _place(rows, "apart", torch.float32)
    want = _norm64(views[0])
    assert abs(float(ddp.GradSet(views).norm()[0]) - want) <= 16 * U * want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[1000, 20], [600_000, 20]])
def test_infinities_and_nans(sizes, dtype):
    rows = _values(4, sizes, 5, 1.0)
    rows[1][1][3] = float("inf")
    rows[2][0][999] = float("nan")
    rows[3][0][0] = float("-inf")
    rows[3][1][19] = float("nan")
    views, _ = _place(rows, "apart", DT[dtype])
    before = [[v.clone() for v in row] for row in views]
    s = ddp.GradSet(views)
    norms = s.norm_clip(1.0).cpu()
    assert math.isfinite(norms[0]) and norms[1] == float("inf") and math.isnan(norms[2]) and math.isnan(norms[3])
    assert bool(torch.isnan(views[1][1][3])) and not bool(views[1][0].any())        # c = 0: inf * 0 is NaN
    assert bool(torch.isnan(views[2][0]).all())
    assert bool(torch.isfinite(views[0][0]).all()) and not torch.equal(views[0][0], before[0][0])


def test_zero_gradients_and_a_limit_that_is_not_reached():
    views, _ = _place([[torch.zeros(4099), torch.zeros(17)]], "odd", torch.float32)
    s = ddp.GradSet(views)
    assert float(s.norm_clip(1.0)[0]) == 0.0
    views[0][0].fill_(-0.0)
    assert float(s.norm_clip(float("inf"))[0]) == 0.0
    assert bool(torch.signbit(views[0][0]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[3000, 500, 5], [700_001, 40_000, 5], [60_000_001]],
                         ids=["cluster", "one_launch", "two_launches"])
def test_norm_does_not_depend_on_the_grid(sizes, dtype):
    if sizes[0] > 10_000_000:
        views = [[torch.randn(n, device="cuda").to(DT[dtype]) for n in sizes] for _ in range(2)]
    else:
        views, _ = _place(_values(2, sizes, 11), "packed", DT[dtype])
    s = ddp.GradSet(views)
    want = s.norm().clone()
    for r in range(2):
        ref = _norm64(views[r])
        assert abs(float(want[r]) - ref) <= 16 * U * ref
    for cap in (1, 3, 15, 150):
        prev = ddp.ddp_set_max_ctas(cap)
        try:
            got = s.norm(out=torch.empty(2, device="cuda"))
            torch.cuda.synchronize()
        finally:
            ddp.ddp_set_max_ctas(prev)
        assert torch.equal(got, want)


@pytest.mark.parametrize("limit", [0.5, 0.1])
@pytest.mark.parametrize("sizes", [[100_000, 333], [3000, 33]])
def test_set_on_another_stream_and_in_a_graph(sizes, limit):
    views, _ = _place(_values(2, sizes, 2), "apart", torch.float32)
    s = ddp.GradSet(views)
    want = s.norm().clone()
    torch.cuda.synchronize()
    q = torch.cuda.Stream()
    out = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    s.norm(out=out, stream=q)
    q.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.norm(out=out)
        s.clip(limit, out)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert k or torch.equal(out, want)
    for r in range(2):
        assert abs(_norm64(views[r]) - min(limit, float(want[r]))) < 1e-5


@pytest.mark.parametrize("sizes", [[100_000, 333], [1 + (37 * i) % 211 for i in range(900)]], ids=["few", "many"])
def test_first_norm_inside_a_capture_then_eager_ones(sizes):
    views, _ = _place(_values(2, sizes, 2), "apart", torch.float32)
    want = ddp.GradSet(views).norm().clone()
    s = ddp.GradSet(views)
    out = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                # the set's first call: its counter is cleared by every replay
        s.norm(out=out)
    assert torch.equal(s.norm(), want)           # and by the first eager call, replayed or not
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(s.norm(), want)


@pytest.mark.parametrize("world,sizes", [(40, [3000, 7]), (17, [200_003]), (300, [50])])
def test_norm_and_clip_of_many_ranks(world, sizes):
    views, held = _place(_values(world, sizes, 13, 1e-2), "apart", torch.float32)
    want = [_norm64(row) for row in views]
    s = ddp.GradSet(views)
    norms = s.norm_clip(want[0]).cpu()
    _check_held(held, "many ranks")
    for r in range(world):
        assert abs(float(norms[r]) - want[r]) <= 16 * U * want[r]
        got, limit = _norm64(views[r]), min(want[r], want[0])
        assert abs(got - limit) <= 16 * U * limit + 2e-6


def test_elements_past_32_bits():
    n = (1 << 31) + 4097
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    s = ddp.GradSet([[g]])
    want = 0.5 * math.sqrt(n)
    got = float(s.norm()[0])
    assert abs(got - want) <= 16 * U * want
    s.clip(want / 4)
    c = torch.tensor(0.125, dtype=torch.bfloat16)
    assert float(g[0]) == float(g[-1]) == float(g[1 << 31]) == float(c)
    assert int((g == c.cuda()).sum()) == n


# --------------------------------------------------------------------------
# The sync that returns the norm
# --------------------------------------------------------------------------

def _sync_views(world, sizes, dtype, seed, layout):
    return _place([[t * 1e-2 for t in row] for row in _values(world, sizes, seed, 1.0)], layout, DT[dtype])


@pytest.mark.parametrize("algo", [ddp.DDP_ALGO_VIEW, ddp.DDP_ALGO_FUSED, ddp.DDP_ALGO_STAGED, ddp.DDP_ALGO_BF16_HOOK,
                                  ddp.DDP_ALGO_BF16_HOOK_VIEW, ddp.DDP_ALGO_FP16_HOOK_VIEW])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("world,sizes,layout", [
    (1, [1000, 3], "apart"), (2, [300_001, 7, 0, 40_000], "packed"), (3, [700_001, 1, 5, 900_000], "apart"),
    (5, [1, 2, 3], "odd"), (8, [400_003, 100_000, 999], "odd"), (8, [400_003, 100_000, 999], "apart"),
    (16, [260_000, 9], "apart"), (2, [6_000_001, 100], "apart"), (33, [50_001], "apart"), (4, [800_001, 5], "packed"),
    (2, [0, 0], "apart"), (150, [3001, 40], "apart"), (2, [1 + (37 * i) % 911 for i in range(700)], "packed"),
])
def test_sync_norm_keeps_the_syncs_bits(world, sizes, layout, dtype, algo):
    hook = algo in (ddp.DDP_ALGO_BF16_HOOK, ddp.DDP_ALGO_BF16_HOOK_VIEW, ddp.DDP_ALGO_FP16_HOOK_VIEW)
    if hook and dtype == "bf16":
        pytest.skip("the hooks take float32 gradients")
    views, held = _sync_views(world, sizes, dtype, 4, layout)
    other, _ = _sync_views(world, sizes, dtype, 4, layout)
    plan = ddp.ddp_plan_buckets(sizes, ddp.BF16 if dtype == "bf16" else ddp.F32, 64 << 10, 1 << 20)
    bt = torch.bfloat16 if algo == ddp.DDP_ALGO_BF16_HOOK else DT[dtype]
    buckets = None
    if algo in (ddp.DDP_ALGO_FUSED, ddp.DDP_ALGO_STAGED, ddp.DDP_ALGO_BF16_HOOK):
        buckets = [[torch.empty(int(n), dtype=bt, device="cuda") for n in plan[2]] for _ in range(world)]
    ddp.ddp_sync_buckets(other, plan, buckets, algo=algo)
    call = ddp.SyncNormCall(views, plan, buckets, algo=algo)
    norms = call()
    torch.cuda.synchronize()
    _check_held(held, "sync norm")
    for r in range(world):
        assert all(torch.equal(a, b) for a, b in zip(views[r], other[r]))
    want = _norm64(views[0])
    assert norms.shape == (world,) and bool((norms == norms[0]).all())
    assert abs(float(norms[0]) - want) <= 16 * U * want


@pytest.mark.parametrize("kernel", [ddp.DDP_FUSED_AUTO, ddp.DDP_FUSED_VECTOR, ddp.DDP_FUSED_TMA])
@pytest.mark.parametrize("cap", [0, 7])
def test_sync_norm_under_other_kernels_and_budgets(kernel, cap):
    world, sizes = 8, [1_000_003, 7, 250_000]
    views, _ = _sync_views(world, sizes, "f32", 6, "apart")
    other, _ = _sync_views(world, sizes, "f32", 6, "apart")
    plan = ddp.ddp_plan_buckets(sizes, ddp.F32)
    ddp.ddp_sync_buckets(other, plan, None, algo=ddp.DDP_ALGO_VIEW)
    call = ddp.SyncNormCall(views, plan)
    k, c = ddp.ddp_set_fused_kernel(kernel), ddp.ddp_set_max_ctas(cap)
    try:
        norms = call()
        torch.cuda.synchronize()
    finally:
        ddp.ddp_set_fused_kernel(k)
        ddp.ddp_set_max_ctas(c)
    assert all(torch.equal(a, b) for x, y in zip(views, other) for a, b in zip(x, y))
    want = _norm64(views[0])
    assert abs(float(norms[0]) - want) <= 16 * U * want


@pytest.mark.parametrize("value,check", [(float("inf"), math.isinf), (float("nan"), math.isnan), (1e25, math.isfinite),
                                         (1e-25, math.isfinite)])
@pytest.mark.parametrize("world,n", [(2, 5000), (4, 600_001)])
def test_sync_norm_of_extreme_values(world, n, value, check):
    views, _ = _sync_views(world, [n, 13], "f32", 9, "apart")
    for row in views:
        row[0].mul_(0.0 if abs(value) < 1 else 1.0)
        row[1].mul_(0.0 if abs(value) < 1 else 1.0)
    views[0][0][n // 2] = value
    plan = ddp.ddp_plan_buckets([n, 13], ddp.F32)
    got = float(ddp.SyncNormCall(views, plan)()[0])
    assert check(got)
    if math.isfinite(got):
        want = _norm64(views[0])
        assert abs(got - want) <= 16 * U * want


# --------------------------------------------------------------------------
# AdamW
# --------------------------------------------------------------------------

def _adamw64(p, m, v, g, c, t, lr, b1, b2, eps, wd):
    """The step in float64 and the tolerances of its three results."""
    p, m, v, g = (x.double() for x in (p, m, v, g))
    gc = c * g
    m2 = b1 * m + (1 - b1) * gc
    v2 = b2 * v + (1 - b2) * gc * gc
    root = torch.sqrt(v2 / (1 - b2 ** t)) + eps
    update = lr / (1 - b1 ** t) * m2 / root
    p2 = p - lr * wd * p - update
    tol_m = 6 * U * ((b1 * m).abs() + ((1 - b1) * gc).abs()) + 2 * TINY
    tol_v = 16 * U * v2 + 4 * TINY
    # v's own error reaches the root: absolutely where v is at the bottom of the range
    slack = torch.sqrt((v2 + tol_v) / (1 - b2 ** t)) - torch.sqrt(v2 / (1 - b2 ** t))
    tol_p = (2 * U * p.abs() + 32 * U * update.abs() + lr / (1 - b1 ** t) * tol_m / root
             + update.abs() * torch.clamp(slack / root, max=1.0) + 2 * TINY)
    return (p2, tol_p), (m2, tol_m), (v2, tol_v)


def _moments(world, sizes, seed, fresh):
    def rows(s, scale, square=False):
        v = _values(world, sizes, s, scale)
        return [[t.square() if square else t for t in row] for row in v]
    zero = [[torch.zeros(n, dtype=torch.float64) for n in sizes] for _ in range(world)]
    return rows(seed, 0.02), (zero if fresh else rows(seed + 1, 1e-3)), (zero if fresh else rows(seed + 2, 1e-3, True))


@pytest.mark.parametrize("dtype,copies", [("f32", False), ("bf16", True), ("f32", True), ("bf16", False)])
@pytest.mark.parametrize("layout", ["apart", "packed", "odd"])
@pytest.mark.parametrize("sizes", ["one", "empty", "some_empty", "edges", "tile", "mixed", "many"])
@pytest.mark.parametrize("t0,clipped", [(0, True), (1000, False)])
def test_adamw(sizes, layout, dtype, copies, t0, clipped):
    if sizes == "many" and (dtype, copies) != ("bf16", True):
        pytest.skip("one combination covers the table's end")
    world = 1 if sizes == "many" else 2
    n = SIZES[sizes]
    hyper = dict(lr=3e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1)
    p, m, v = _moments(world, n, 21, t0 == 0)
    (p, hp), (m, hm), (v, hv) = (_place(x, layout, torch.float32) for x in (p, m, v))
    g, hg = _place(_values(world, n, 30), layout, DT[dtype])
    c, hc = _place([[torch.zeros(k) for k in n] for _ in range(world)], layout, torch.bfloat16) if copies else (None, [])
    no_decay = [i % 3 == 1 for i in range(len(n))]
    steps = torch.full((world,), t0, dtype=torch.int32, device="cuda")
    norms = torch.tensor([2.5, 0.25][:world], device="cuda")
    opt = ddp.AdamW(p, g, m, v, copies=c, no_decay=no_decay, steps=steps)
    for k in range(2):                                   # the second step starts from the first one's results
        old = [[[t.clone() for t in row] for row in x] for x in (p, m, v, g)]
        opt.step(hyper["lr"], (hyper["b1"], hyper["b2"]), hyper["eps"], hyper["wd"], norms if clipped else None, 1.0)
        torch.cuda.synchronize()
        assert steps.tolist() == [t0 + k + 1] * world
        for r in range(world):
            cf = min(1.0, 1.0 / (float(norms[r]) + 1e-6)) if clipped else 1.0
            for i in range(len(n)):
                want = _adamw64(*[old[j][r][i] for j in range(4)], cf, t0 + k + 1, hyper["lr"], hyper["b1"], hyper["b2"],
                                hyper["eps"], 0.0 if no_decay[i] else hyper["wd"])
                for x, (y, tol), what in zip((p, m, v), want, "pmv"):
                    d = (x[r][i].double() - y).abs()
                    assert bool((d <= tol).all()), (what, r, i, float((d / tol).max()))
                assert torch.equal(g[r][i], old[3][r][i]), "a gradient was written"
                if copies:
                    assert torch.equal(c[r][i], p[r][i].bfloat16())
    for held in (hp, hm, hv, hg, hc):
        if held is not hc or copies:
            _check_held(held, "adamw")


def test_adamw_arrays_of_unlike_alignment():
    n = 10_007
    base = {k: torch.randn(n + 8, device="cuda") for k in "pgm"}
    base["v"] = torch.rand(n + 8, device="cuda")
    for shift in ((0, 1, 2, 3), (1, 1, 1, 2), (3, 3, 3, 3), (2, 0, 2, 2)):
        p, g, m, v = (base[k].clone()[s:s + n] for k, s in zip("pgmv", shift))
        old = [t.clone() for t in (p, m, v, g)]
        ddp.AdamW([[p]], [[g]], [[m]], [[v]]).step(1e-3)
        want = _adamw64(*old, 1.0, 1, 1e-3, 0.9, 0.999, 1e-8, 0.0)
        for x, (y, tol) in zip((p, m, v), want):
            assert bool(((x.double() - y).abs() <= tol).all()), shift


@pytest.mark.parametrize("beta", [(0.0, 0.0), (0.9, 0.95), (0.9999, 0.99999)])
@pytest.mark.parametrize("t0", [0, 1, 9, 100_000, 20_000_000])
def test_adamw_bias_corrections(t0, beta):
    n = 5000
    p, m, v, g = (torch.randn(n, device="cuda") * s for s in (0.02, 1e-3, 1e-3, 1e-2))
    v = v.square()
    old = [t.clone() for t in (p, m, v, g)]
    steps = torch.full((1,), t0, dtype=torch.int32, device="cuda")
    ddp.AdamW([[p]], [[g]], [[m]], [[v]], steps=steps).step(1e-3, beta, 1e-8, 0.01)
    want = _adamw64(*old, 1.0, t0 + 1, 1e-3, beta[0], beta[1], 1e-8, 0.01)
    for x, (y, tol) in zip((p, m, v), want):
        assert bool(((x.double() - y).abs() <= tol).all())


def test_many_tensors_through_changing_calls_and_a_graph():
    """Tables that one launch's parameters do not take: captured before and after the other kernel's runs."""
    world, sizes = 3, [1 + (37 * i) % 911 for i in range(500)]
    plan = ddp.ddp_plan_buckets(sizes, ddp.F32, 64 << 10, 256 << 10)
    views, held = _place([[t * 1e-2 for t in row] for row in _values(world, sizes, 4, 1.0)], "apart", torch.float32)
    first = [[t.clone() for t in row] for row in views]

    def reset():
        for row, old in zip(views, first):
            for t, o in zip(row, old):
                t.copy_(o)
    other, _ = _place([[t * 1e-2 for t in row] for row in _values(world, sizes, 4, 1.0)], "apart", torch.float32)
    ddp.ddp_sync_buckets(other, plan, None, algo=ddp.DDP_ALGO_VIEW)
    want = _norm64(other[0])
    call = ddp.SyncNormCall(views, plan)

    def check(norms):
        torch.cuda.synchronize()
        _check_held(held, "many tensors")
        assert all(torch.equal(a, b) for x, y in zip(views, other) for a, b in zip(x, y))
        assert bool(((norms.double() - want).abs() <= 16 * U * want).all())
    check(call())
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cap in (7, 0):                                   # below four CTAs an SM: the sync's own kernels, then a norm pass
        reset()
        prev = ddp.ddp_set_max_ctas(cap)
        try:
            check(call())
        finally:
            ddp.ddp_set_max_ctas(prev)
        reset()
        graph.replay()
        check(call.norms)


def _rows(world, count, size, seed, dtype=torch.float32, std=1.0):
    """[world, count, size rounded up] with zeros past size, and its tensors as views."""
    width = -(-size // 64) * 64
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(world, count, width, dtype=dtype, device="cuda")
    x[:, :, :size].normal_(0.0, std, generator=g)
    return x, [[x[r, i, :size] for i in range(count)] for r in range(world)]


def test_lists_that_take_several_launches_of_their_own():
    """More tensors than one launch's table takes, and too much data for a table in device memory."""
    x, views = _rows(1, 1200, 120_001, 3)                # 2 launches of ranges, 576 MB
    want = float(x.double().square().sum().sqrt())
    s = ddp.GradSet(views)
    got = float(s.norm()[0])
    assert abs(got - want) <= 16 * U * want
    y = x.double() * min(1.0, 0.25 * want / (got + 1e-6))
    s.clip(0.25 * want)
    assert bool(((x.double() - y).abs() <= 4 * U * y.abs() + TINY).all())
    del s, x, y, views
    x, views = _rows(2, 310, 110_001, 4)                 # 2 launches of members, 546 MB moved
    other = x.clone()
    theirs = [[other[r, i, :110_001] for i in range(310)] for r in range(2)]
    plan = ddp.ddp_plan_buckets([110_001] * 310, ddp.F32)
    ddp.ddp_sync_buckets(theirs, plan, None, algo=ddp.DDP_ALGO_VIEW)
    norms = ddp.SyncNormCall(views, plan)()
    assert torch.equal(x, other)
    want = float(other[0].double().square().sum().sqrt())
    assert bool(((norms.double() - want).abs() <= 16 * U * want).all())
    del x, other, views, theirs
    p, pv = _rows(1, 600, 40_001, 5, std=0.02)           # 2 launches of items, 672 MB
    g, gv = _rows(1, 600, 40_001, 6, std=1e-2)
    m, mv = _rows(1, 600, 40_001, 7, std=1e-3)
    v, vv = _rows(1, 600, 40_001, 8, std=1e-3)
    v.square_()
    old = [t.clone() for t in (p, m, v, g)]
    opt = ddp.AdamW(pv, gv, mv, vv, steps=torch.full((1,), 9, dtype=torch.int32, device="cuda"))
    opt.step(1e-3, weight_decay=0.1)
    assert opt.steps.tolist() == [10]
    for t, (want, tol) in zip((p, m, v), _adamw64(*old, 1.0, 10, 1e-3, 0.9, 0.999, 1e-8, 0.1)):
        assert bool(((t.double() - want).abs() <= tol).all())


def test_adamw_skips_ranks_whose_norm_is_not_finite():
    world, n = 4, 9001
    p, g, m, v = ([[torch.rand(n, device="cuda")] for _ in range(world)] for _ in range(4))
    old = [[row[0].clone() for row in x] for x in (p, m, v)]
    norms = torch.tensor([1.0, float("inf"), float("nan"), 3e38], device="cuda")
    opt = ddp.AdamW(p, g, m, v)
    for k in range(2):
        opt.step(1e-3, norms=norms, max_norm=1.0)
    assert opt.steps.tolist() == [2, 0, 0, 2]
    for r in range(world):
        same = [torch.equal(x[r][0], o[r]) for x, o in zip((p, m, v), old)]
        assert same == [r in (1, 2)] * 3 if r != 3 else not same[1]


def test_adamw_zero_gradients_and_a_shared_gradient():
    n, world = 4097, 3
    g = torch.zeros(n, device="cuda")
    p, m, v = ([[torch.zeros(n, device="cuda")] for _ in range(world)] for _ in range(3))
    opt = ddp.AdamW(p, [[g]] * world, m, v)              # every rank reads the one averaged gradient
    opt.step(1e-2)
    assert not any(bool(x[r][0].any()) for x in (p, m, v) for r in range(world))
    g.fill_(2.0)
    opt.step(1e-2)
    torch.cuda.synchronize()
    assert all(torch.equal(p[0][0], p[r][0]) for r in range(world)) and bool((p[0][0] < 0).all())


def test_adamw_results_do_not_depend_on_the_grid_and_replay_in_a_graph():
    n = [300_001, 17]
    runs = []
    for cap in (0, 1, 37):
        gen = torch.Generator(device="cuda").manual_seed(1)
        p, g, m, v = ([[torch.rand(k, device="cuda", generator=gen) for k in n] for _ in range(2)] for _ in range(4))
        opt = ddp.AdamW(p, g, m, v)
        prev = ddp.ddp_set_max_ctas(cap)
        try:
            for _ in range(4):
                opt.step(1e-3, weight_decay=0.1)
            torch.cuda.synchronize()
        finally:
            ddp.ddp_set_max_ctas(prev)
        assert opt.steps.tolist() == [4, 4]
        runs.append([t for x in (p, m, v) for row in x for t in row])
    gen = torch.Generator(device="cuda").manual_seed(1)
    p, g, m, v = ([[torch.rand(k, device="cuda", generator=gen) for k in n] for _ in range(2)] for _ in range(4))
    opt = ddp.AdamW(p, g, m, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(1e-3, weight_decay=0.1)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    runs.append([t for x in (p, m, v) for row in x for t in row])
    assert opt.steps.tolist() == [4, 4]
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_adamw_elements_past_32_bits():
    n = (1 << 31) + 4099
    p = torch.full((n,), 1.0, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    ddp.AdamW([[p]], [[g]], [[m]], [[v]]).step(0.25)
    torch.cuda.synchronize()
    first = float(p[0])
    assert abs(first - 0.75) < 1e-6
    assert int((p == first).sum()) == n and float(m[-1]) == float(m[0]) and float(v[1 << 31]) == float(v[0])


def test_adamw_step_refusals():
    p, g, m, v = ([[torch.ones(8, device="cuda")]] for _ in range(4))
    opt = ddp.AdamW(p, g, m, v)
    norms = torch.ones(1, device="cuda")
    nan, inf = float("nan"), float("inf")
    for kw in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(betas=(1.0, 0.9)), dict(betas=(0.9, 1.0)),
               dict(betas=(-0.1, 0.9)), dict(betas=(nan, 0.9)), dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-60),
               dict(weight_decay=-0.1), dict(weight_decay=inf), dict(norms=norms), dict(norms=norms, max_norm=-1.0),
               dict(norms=norms, max_norm=nan), dict(norms=m[0][0][:1], max_norm=1.0)):
        with pytest.raises(ddp.DDPError) as e:
            opt.step(**{"lr": 1e-3, **kw})
        assert e.value.status == -1, kw
    with pytest.raises(ValueError):
        opt.step(1e-3, norms=torch.ones(2, device="cuda"), max_norm=1.0)
    torch.cuda.synchronize()
    assert opt.steps.tolist() == [0] and float(p[0][0].sum()) == 8.0


def test_a_training_step_end_to_end():
    """Backward's gradients -> sync with the norm -> clipped update: every rank keeps the same weights, and they are
    those of float64 arithmetic on the averaged gradients."""
    numels = workloads.param_numels(workloads.decoder_param_shapes(n_layer=2, d_model=64, d_ff=256, vocab=500, n_pos=32))
    world = 4
    p0 = _values(1, numels, 40, 0.02)[0]
    p, _ = _place([p0] * world, "apart", torch.float32)
    m, _ = _place([[torch.zeros(k) for k in numels]] * world, "apart", torch.float32)
    v, _ = _place([[torch.zeros(k) for k in numels]] * world, "apart", torch.float32)
    g, _ = _place(_values(world, numels, 50, 1.0), "packed", torch.float32)
    plan = ddp.ddp_plan_buckets(numels, ddp.F32, 64 << 10, 256 << 10)
    sync, opt = ddp.SyncNormCall(g, plan), ddp.AdamW(p, g, m, v)
    ref = [[t.double().clone() for t in row] for row in (p[0], m[0], v[0])]
    for t in (1, 2):
        for r, row in enumerate(_values(world, numels, 50 + t, 1.0)):
            for a, b in zip(g[r], row):
                a.copy_(b.float())
        mean = [sum(g[r][i].double() for r in range(world)) / world for i in range(len(numels))]
        opt.step(1e-3, weight_decay=0.1, norms=sync(), max_norm=1.0)
        torch.cuda.synchronize()
        c = min(1.0, 1.0 / (_norm64(mean) + 1e-6))
        for i in range(len(numels)):
            ref[1][i] = 0.9 * ref[1][i] + 0.1 * c * mean[i]
            ref[2][i] = 0.999 * ref[2][i] + 0.001 * (c * mean[i]) ** 2
            ref[0][i] -= 1e-3 * (0.1 * ref[0][i] + ref[1][i] / (1 - 0.9 ** t)
                                 / (torch.sqrt(ref[2][i] / (1 - 0.999 ** t)) + 1e-8))
    for r in range(world):
        for i in range(len(numels)):
            assert torch.equal(p[r][i], p[0][i])
            assert float((p[r][i].double() - ref[0][i]).abs().max()) < 1e-6


def test_the_example_trains_and_its_ranks_agree():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, norms, params = example.train(ranks=3, steps=60)
    assert losses[-1] < 0.5 * losses[0] and all(math.isfinite(n) and n > 0 for n in norms)
    for row in params[1:]:
        assert all(torch.equal(a, b) for a, b in zip(row, params[0]))
