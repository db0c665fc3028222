"""Refusals of the gradient norm, clipping, norm-in-sync and AdamW entry points.

Every call here is refused by the host checks (or makes a set, which makes no
CUDA call), so no made-up pointer reaches the GPU.
"""
import ctypes

import pytest
import torch

import gradient_sync_plan_gb300 as ddp

H = 0x7f0000000000                     # made-up device addresses, never dereferenced
WS = H + (1 << 40)
NORMS = H + (1 << 41)
FREE = H + (1 << 42)
INF, NAN = float("inf"), float("nan")


def _vp(*p):
    return (ctypes.c_void_p * max(len(p), 1))(*p)


def _i64(*v):
    return (ctypes.c_int64 * max(len(v), 1))(*v)


def _create(world, ptrs, sizes, dtype=0, ws=WS, ws_bytes=None, out=True):
    h = ctypes.c_void_p(1)
    n = 1 << 30 if ws_bytes is None else ws_bytes
    st = ddp.lib().ddp_grad_set_create(world, len(sizes), _vp(*ptrs), _i64(*sizes), dtype, ws, n,
                                       ctypes.byref(h) if out else None)
    assert not out or st == 0 or h.value is None
    return st, h


@pytest.mark.parametrize("want,kw", [
    (-1, dict(world=0)), (-5, dict(world=513)), (-1, dict(dtype=7)), (-1, dict(sizes=[8, -1])),
    (-5, dict(sizes=[8, ddp.MAX_NUMEL + 1], ws_bytes=1 << 60)), (-1, dict(ptrs=[H, None])),
    (-2, dict(ptrs=[H + 2, H + 4096])), (-2, dict(ptrs=[H + 1, H + 4096], dtype=1)), (-1, dict(ptrs=[H, H + 28])),
    (-1, dict(ws=None)), (-2, dict(ws=WS + 8)), (-5, dict(ws_bytes=7)), (-1, dict(ws=H + 16)), (-1, dict(out=False)),
])
def test_grad_set_refusals(want, kw):
    args = dict(world=1, ptrs=[H, H + 4096], sizes=[8, 8])
    args.update(kw)
    assert _create(**args)[0] == want


def test_grad_set_sizes_that_overflow_are_refused():
    L, out = ddp.lib(), ctypes.c_int64(-1)
    for n in ((1 << 62) + 16, (1 << 63) - 1, ddp.MAX_NUMEL + 1):
        assert L.ddp_grad_set_workspace_bytes(1, 1, _i64(n), 0, ctypes.byref(out)) == -5
        assert L.ddp_sync_norm_workspace_bytes(1, 1, _i64(n), 0, ctypes.byref(out)) == -5
    for sizes in ([ddp.MAX_NUMEL, 1], [ddp.MAX_NUMEL] * 3):      # one rank's elements together
        assert L.ddp_grad_set_workspace_bytes(1, len(sizes), _i64(*sizes), 0, ctypes.byref(out)) == -5
        assert L.ddp_sync_norm_workspace_bytes(1, len(sizes), _i64(*sizes), 0, ctypes.byref(out)) == -5
    assert out.value == -1
    assert L.ddp_grad_set_workspace_bytes(1, 1, None, 0, ctypes.byref(out)) == -1
    assert L.ddp_grad_set_workspace_bytes(1, -1, _i64(1), 0, ctypes.byref(out)) == -1
    assert L.ddp_grad_set_workspace_bytes(1, 1, _i64(1), 0, None) == -1
    assert L.ddp_sync_norm_workspace_bytes(1, 1, _i64(1), 0, None) == -1


def test_grad_set_takes_empty_tensors_without_pointers():
    st, h = _create(2, [H, None, H + 4096, None], [8, 0])
    assert st == 0 and ddp.lib().ddp_grad_set_destroy(h) == 0
    assert ddp.lib().ddp_grad_set_destroy(None) == 0


def test_norm_and_clip_refusals():
    L = ddp.lib()
    st, h = _create(2, [H, H + 4096, H + 8192, H + 16384], [8, 8])
    assert st == 0
    for norms, want in ((None, -1), (NORMS + 2, -2), (H + 4096 + 28, -1), (H - 4, -1), (WS, -1)):
        assert L.ddp_grad_norm(h, norms, None) == want
        assert L.ddp_grad_clip(h, norms, 1.0, None) == want
        assert L.ddp_grad_norm_clip(h, norms, 1.0, None) == want
    for bad in (0.0, -1.0, NAN, 1e-60):
        assert L.ddp_grad_clip(h, NORMS, bad, None) == -1
        assert L.ddp_grad_norm_clip(h, NORMS, bad, None) == -1
    assert L.ddp_grad_norm(None, NORMS, None) == -1
    assert L.ddp_grad_clip(None, NORMS, 1.0, None) == -1
    assert L.ddp_grad_norm_clip(None, NORMS, 1.0, None) == -1
    L.ddp_grad_set_destroy(h)


def _sync(world=2, grads=(H, H + 4096), dtype=0, divisor=2, algo=ddp.DDP_ALGO_VIEW, ws=WS, ws_bytes=1 << 20, numel=(8,),
          bucket=(0,), offset=(0,), bucket_numel=(8,), buckets=None, table=True, out=True):
    h, n = ctypes.c_void_p(1), len(numel)
    st = ddp.lib().ddp_sync_norm_create(world, n, _vp(*grads) if table else None, _i64(*numel),
                                        (ctypes.c_int32 * n)(*bucket), _i64(*offset), len(bucket_numel),
                                        _i64(*bucket_numel), None if buckets is None else _vp(*buckets), dtype, divisor,
                                        algo, ws, ws_bytes, ctypes.byref(h) if out else None)
    assert not out or st == 0 or h.value is None
    return st, h


@pytest.mark.parametrize("want,kw", [
    (-1, dict(world=0)), (-5, dict(world=513)), (-1, dict(dtype=5)), (-1, dict(divisor=-1)), (-1, dict(out=False)),
    (-1, dict(ws=None)), (-2, dict(ws=WS + 8)), (-5, dict(ws_bytes=8)), (-1, dict(ws=H + 4096)), (-1, dict(table=False)),
    (-1, dict(algo=ddp.DDP_ALGO_DRYRUN)), (-1, dict(algo=99)), (-1, dict(algo=ddp.DDP_ALGO_FUSED)),
    (-1, dict(algo=ddp.DDP_ALGO_BF16_HOOK_VIEW, dtype=1)), (-1, dict(numel=(9,))), (-1, dict(numel=(-1,))),
    (-1, dict(offset=(1,))), (-1, dict(offset=(-1,))), (-1, dict(bucket=(1,))), (-1, dict(bucket=(-1,))),
    (-5, dict(bucket_numel=(ddp.MAX_NUMEL + 1,))), (-1, dict(bucket_numel=(-1,))),
    (-1, dict(grads=(H, H + 16))), (-1, dict(grads=(H, None))), (-2, dict(grads=(H, H + 4098))),
    (-1, dict(grads=(H, H + 64, H + 4096, H + 8192), numel=(8, 8), bucket=(0, 0), offset=(0, 7), bucket_numel=(16,))),
    (-1, dict(algo=ddp.DDP_ALGO_FUSED, buckets=(H + (1 << 20), None))),
    (-1, dict(algo=ddp.DDP_ALGO_FUSED, buckets=(H + (1 << 20), H + 16))),
    (-2, dict(algo=ddp.DDP_ALGO_FUSED, buckets=(H + (1 << 20), H + (2 << 20) + 2))),
])
def test_sync_norm_create_refusals(want, kw):
    assert _sync(**kw)[0] == want


def test_sync_norm_run_refusals():
    L = ddp.lib()
    st, h = _sync()
    assert st == 0
    for norms, want in ((None, -1), (NORMS + 1, -2), (H + 28, -1), (H + 4096 - 4, -1), (WS, -1)):
        assert L.ddp_sync_norm_run(h, norms, None) == want
    assert L.ddp_sync_norm_run(None, NORMS, None) == -1
    assert L.ddp_sync_norm_destroy(h) == 0 and L.ddp_sync_norm_destroy(None) == 0


def _adamw(world=1, n=1, p=(H,), g=(H + (1 << 20),), m=(H + (2 << 20),), v=(H + (3 << 20),), c=None, sizes=(8,),
           dtype=0, steps=NORMS, ws=WS, ws_bytes=1 << 20, out=True):
    h = ctypes.c_void_p(1)
    tab = [None if t is None else _vp(*t) for t in (p, g, m, v, c)]
    st = ddp.lib().ddp_adamw_create(world, n, tab[0], tab[1], dtype, tab[2], tab[3], tab[4], _i64(*sizes), None, steps,
                                    ws, ws_bytes, ctypes.byref(h) if out else None)
    assert not out or st == 0 or h.value is None
    return st, h


@pytest.mark.parametrize("want,kw", [
    (-5, dict(ws_bytes=256)), (-1, dict(world=0)), (-5, dict(world=513)), (-1, dict(n=-1)), (-1, dict(sizes=(-1,))), (-1, dict(dtype=2)),
    (-5, dict(sizes=(ddp.MAX_NUMEL + 1,))), (-1, dict(out=False)), (-1, dict(steps=None)), (-2, dict(steps=NORMS + 2)),
    (-1, dict(ws=None)), (-2, dict(ws=WS + 8)), (-1, dict(ws=NORMS)),
    (-1, dict(p=None)), (-1, dict(g=None)), (-1, dict(m=None)), (-1, dict(v=None)),
    (-1, dict(p=(None,))), (-1, dict(g=(None,))), (-1, dict(m=(None,))), (-1, dict(v=(None,))), (-1, dict(c=(None,))),
    (-2, dict(p=(H + 2,))), (-2, dict(g=(H + 2,))), (-2, dict(m=(H + 1,))), (-2, dict(v=(H + 2,))), (-2, dict(c=(H + (4 << 20) + 1,))),
    (-1, dict(m=(H + 28,))), (-1, dict(v=(H + (2 << 20) + 4,))), (-1, dict(g=(H + 16,))), (-1, dict(c=(H + 4,))),
    (-1, dict(steps=H)), (-1, dict(ws=H + 16)),
])
def test_adamw_refusals(want, kw):
    assert _adamw(**kw)[0] == want


def test_adamw_step_refusals():
    L = ddp.lib()
    st, h = _adamw()
    assert st == 0
    good = dict(lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1, norms=None, max_norm=0.0)
    for kw in (dict(lr=-1.0), dict(lr=NAN), dict(lr=INF), dict(b1=1.0), dict(b2=1.0), dict(b1=-0.1), dict(b1=NAN),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-60), dict(eps=NAN), dict(wd=-0.1), dict(wd=INF),
               dict(norms=FREE), dict(norms=FREE, max_norm=-1.0), dict(norms=FREE, max_norm=NAN),
               dict(norms=H, max_norm=1.0), dict(norms=NORMS, max_norm=1.0)):
        a = {**good, **kw}
        assert L.ddp_adamw_step(h, a["lr"], a["b1"], a["b2"], a["eps"], a["wd"], a["norms"], a["max_norm"], None) == -1, kw
    assert L.ddp_adamw_step(h, 1e-3, 0.9, 0.999, 1e-8, 0.0, FREE + 2, 1.0, None) == -2
    L.ddp_adamw_destroy(h)


def test_adamw_step_and_destroy_without_a_handle():
    L = ddp.lib()
    assert L.ddp_adamw_step(None, 1e-3, 0.9, 0.999, 1e-8, 0.0, None, 0.0, None) == -1
    assert L.ddp_adamw_destroy(None) == 0


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros(2, 8)
    rows = [[x[0, :4]], [x[1, :4]]]
    for make in (lambda: ddp.GradSet(rows), lambda: ddp.AdamW(rows, rows, rows, rows)):
        with pytest.raises(ValueError, match="device memory"):
            make()
    with pytest.raises(ValueError, match="contiguous"):
        ddp.GradSet([[x.t()]])
    with pytest.raises(ValueError, match="contiguous"):
        ddp.GradSet([[x.double()]])
    plan = ddp.ddp_plan_buckets([4], ddp.F32)
    with pytest.raises(ValueError, match="device memory"):
        ddp.SyncNormCall(rows, plan)
