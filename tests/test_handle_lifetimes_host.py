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
    plain = ddp._stream
    monkeypatch.setattr(ddp, "_stream", lambda s: 0 if s is None else plain(s))      # no current stream here


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


# --------------------------------------------------------------------------
# Streams of a handle's own memory
# --------------------------------------------------------------------------

class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class _Library:
    """Entry points that launch nothing."""
    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture
def recorded(cpu_tensors, monkeypatch):
    """{stream handle: [addresses recorded with it]}, and the current stream's handle to be set."""
    log, current = {}, {"handle": 0}
    plain = ddp._stream
    monkeypatch.setattr(ddp, "_stream", lambda s: current["handle"] if s is None else plain(s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream(current["handle"]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _Stream(handle))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: log.setdefault(s.cuda_stream, []).append(t.data_ptr()))
    return log, current


def _calls(kind, handle):
    """Every call of a handle that launches work, as functions of stream."""
    if kind == "grad_set":
        return [lambda s: handle.norm(stream=s), lambda s: handle.clip(1.0, stream=s),
                lambda s: handle.norm_clip(1.0, stream=s)]
    if kind == "sync_norm":
        return [lambda s: handle(s)]
    return [lambda s: handle.step(1e-3, stream=s)]


@pytest.mark.parametrize("number", range(3))
@pytest.mark.parametrize("kind", ["grad_set", "sync_norm", "adamw"])
def test_a_call_on_another_stream_is_recorded_with_the_handles_memory(kind, number, recorded):
    """The allocator may give a block out again, in the order of the stream it was allocated on, as soon as its tensor
    is gone: it has to know of every other stream that works on it."""
    log, current = recorded
    handle, _ = _made(kind)
    handle._lib = _Library()
    calls = _calls(kind, handle)
    call = calls[number % len(calls)]
    own = {handle._workspace.data_ptr(), (handle.steps if kind == "adamw" else handle.norms).data_ptr()}
    call(None)
    call(_Stream(0))
    assert not log, "nothing to record on the stream that the memory comes from"
    call(_Stream(4096))
    assert set(log) == {4096} and set(log[4096]) == own
    call(8192)                                   # a plain handle
    assert set(log) == {4096, 8192} and set(log[8192]) == own
    current["handle"] = 12288                    # the current stream has changed since
    call(None)
    assert set(log) == {4096, 8192, 12288} and set(log[12288]) == own
    for s in (None, 0, 4096, 8192, _Stream(8192)):
        call(s)
    assert all(len(v) == len(own) for v in log.values()) and set(log) == {4096, 8192, 12288}, "once a stream is enough"


@pytest.mark.parametrize("handle_of_default", [0, 1])
def test_the_default_stream_as_a_plain_handle(handle_of_default, recorded):
    log, current = recorded
    current["handle"] = 4096
    handle, _ = _made("grad_set")
    handle._lib = _Library()
    handle.norm(stream=handle_of_default)
    assert set(log) == {0} and len(log[0]) == 2


def test_step_counts_of_the_caller_are_the_callers(recorded):
    log, _ = recorded
    steps = torch.zeros(2, dtype=torch.int32)
    opt = ddp.AdamW(*(_rows() for _ in range(4)), steps=steps)
    opt._lib = _Library()
    opt.step(1e-3, stream=4096)
    assert log == {4096: [opt._workspace.data_ptr()]}
