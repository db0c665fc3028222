"""What the binding's handles keep alive and what they tell the allocator, without a GPU.

The library reads no memory when a handle is made, so CPU tensors stand in for
device tensors where the binding's own memory check is taken out.
"""
import gc
import weakref

import pytest
import torch

import gradient_sync_plan_gb300 as ddp


@pytest.fixture
def cpu_tensors(monkeypatch):
    monkeypatch.setattr(ddp, "_check_memory", lambda t, memory, what: None)


def _rows(world=2, sizes=(8, 5), dtype=torch.float32):
    return [[torch.zeros(n, dtype=dtype) for n in sizes] for _ in range(world)]


def _made(kind):
    """(handle, lists it was given)"""
    plan = ddp.ddp_plan_buckets([8, 5], ddp.F32)
    if kind == "grad_set":
        lists = [_rows()]
        return ddp.GradSet(lists[0]), lists
    if kind == "adamw":
        lists = [_rows() for _ in range(4)] + [_rows(dtype=torch.bfloat16)]
        return ddp.AdamW(*lists[:4], copies=lists[4]), lists
    lists = [_rows(), [[torch.zeros(int(n)) for n in plan[2]] for _ in range(2)]]
    if kind == "sync_norm":
        return ddp.SyncNormCall(lists[0], plan, lists[1], algo=ddp.DDP_ALGO_FUSED), lists
    if kind == "sync":
        return ddp.SyncCall(lists[0], plan, lists[1]), lists
    return ddp.Reducer(lists[0], plan, lists[1], algo=ddp.DDP_ALGO_DRYRUN), lists


KINDS = ["grad_set", "adamw", "sync_norm", "sync", "reducer"]


@pytest.mark.parametrize("kind", KINDS)
def test_handles_keep_the_tensors_whose_addresses_they_hold(kind, cpu_tensors):
    """A program that puts new tensors into the lists it passed (as autograd's results) must not free the old ones."""
    handle, lists = _made(kind)
    held = [weakref.ref(t) for rows in lists for row in rows for t in row]
    for rows in lists:
        for row in rows:
            row[:] = [torch.ones_like(t) for t in row]
        rows.clear()
    gc.collect()
    assert all(r() is not None for r in held)
    del handle
    gc.collect()
    assert not any(r() is not None for r in held), "a handle that is gone keeps nothing"


def test_a_handle_keeps_the_step_counts_it_was_made_with(cpu_tensors):
    steps = torch.zeros(2, dtype=torch.int32)
    opt = ddp.AdamW(*(_rows() for _ in range(4)), steps=steps)
    held = weakref.ref(steps)
    opt.steps = steps = None
    gc.collect()
    assert held() is not None
