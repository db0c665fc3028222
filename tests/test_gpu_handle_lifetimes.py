"""A handle that goes while a call on another stream still works on its memory."""
import pytest
import torch

import gradient_sync_plan_gb300 as ddp

pytestmark = pytest.mark.gpu

SIZES = [1000, 333]


def _rows(world, value=None, dtype=torch.float32):
    rows = [[torch.randn(n, device="cuda").to(dtype) for n in SIZES] for _ in range(world)]
    if value is not None:
        for row in rows:
            for t in row:
                t.fill_(value)
    return rows


def _handle(kind):
    """(handle, the call, tensors of its own)"""
    if kind == "grad_set":
        h = ddp.GradSet(_rows(2))
        return h, lambda q: h.norm_clip(1.0, stream=q)
    if kind == "sync_norm":
        h = ddp.SyncNormCall(_rows(2), ddp.ddp_plan_buckets(SIZES, ddp.F32))
        return h, lambda q: h(q)
    h = ddp.AdamW(_rows(2), _rows(2), _rows(2, 0.0), _rows(2, 0.0))
    return h, lambda q: h.step(1e-3, stream=q)


def _blocks(sizes):
    """Addresses that new tensors of these byte sizes get on the current stream, 64 of each."""
    made = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(64)]
    return {t.data_ptr() for t in made}


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("kind", ["grad_set", "sync_norm", "adamw"])
def test_its_memory_is_not_given_out_before_the_call_is_over(kind, as_handle):
    handle, call = _handle(kind)
    own = [handle._workspace, handle.steps if kind == "adamw" else handle.norms]
    sizes = [t.numel() * t.element_size() for t in own]
    addresses = {t.data_ptr() for t in own}
    keep = handle._keep
    q = torch.cuda.Stream()
    _handle(kind)[1](None)                       # the first launch of a kernel loads it, and waits for the GPU
    _blocks(sizes)
    torch.cuda.synchronize()
    with torch.cuda.stream(q):
        torch.cuda._sleep(400_000_000)           # some 0.2 s before the call starts
    done = torch.cuda.Event()
    result = call(q.cuda_stream if as_handle else q)
    done.record(q)
    del handle, call, own, result
    taken = _blocks(sizes)
    assert not done.query(), "the call was over before the memory was asked for"
    assert not taken & addresses
    torch.cuda.synchronize()
    assert taken and keep


def test_calls_on_another_stream_agree_with_the_creating_ones():
    torch.manual_seed(0)
    q = torch.cuda.Stream()
    plan = ddp.ddp_plan_buckets(SIZES, ddp.F32)
    results = []
    for stream in (None, q):
        torch.manual_seed(1)
        g, p, m, v = _rows(2), _rows(2), _rows(2, 0.0), _rows(2, 0.0)
        sync, opt = ddp.SyncNormCall(g, plan), ddp.AdamW(p, g, m, v)
        torch.cuda.synchronize()                 # the handles' memory and the tensors are there
        for _ in range(3):
            opt.step(1e-2, weight_decay=0.1, norms=sync(stream), max_norm=0.5, stream=stream)
        torch.cuda.synchronize()
        results.append([sync.norms, opt.steps] + [t for rows in (g, p, m, v) for row in rows for t in row])
    assert results[1][1].tolist() == [3, 3]
    assert all(torch.equal(a, b) for a, b in zip(*results))
