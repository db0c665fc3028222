"""Calls of the loss head that follow each other closely: every one ends, and repeats its bits."""
import time

import pytest
import torch

import gradient_sync_plan_gb300 as ddp

pytestmark = pytest.mark.gpu


def _inputs(tokens, vocab, dim, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(device="cuda", generator=gen)
    weights = [(torch.randn(vocab, dim, **kw) * dim ** -0.5).to(dtype) for _ in tokens]
    targets = [torch.randint(0, vocab, (n,), **kw) for n in tokens]
    return weights, [torch.randn(n, dim, **kw).to(dtype) for n in tokens], targets


class Rank:
    def __init__(self, tokens, vocab, dim, dtype, seed):
        weights, self.hidden, self.targets = _inputs(tokens, vocab, dim, dtype, seed)
        self.gw, self.gh = [torch.empty_like(w) for w in weights], [torch.empty_like(h) for h in self.hidden]
        self.head = ddp.LossHead(weights, self.gw, max_tokens=max(tokens))
        self.stream = torch.cuda.Stream()

    def call(self, stream=None):
        self.head.cross_entropy_grad(self.hidden, self.targets, self.gh, stream=stream)

    def results(self):
        return [t.clone() for t in self.gw + self.gh + [self.head.loss]]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,tokens,vocab,dim", [(torch.bfloat16, [1024], 3001, 320), (torch.float32, [1024, 900], 2500, 1100),
                                                    (torch.bfloat16, [2048, 2000], 1030, 64)])
def test_two_heads_of_many_tokens_on_two_streams(dtype, tokens, vocab, dim):
    ranks = [Rank(tokens, vocab, dim, dtype, k) for k in range(2)]
    want = []
    for r in ranks:
        r.call()
        torch.cuda.synchronize()
        want.append(r.results())
    for _ in range(10):
        for r in ranks:
            r.call(stream=r.stream)
    torch.cuda.synchronize()
    assert all(_same(r.results(), w) for r, w in zip(ranks, want))
    assert ddp.ddp_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_call_after_another(dtype):
    # the decoder's head over two ragged ranks: its hidden states' gradients have a depth of many parts in float32
    rank = Rank([1024, 900], 50257, 1024, dtype, 5)
    rank.call()
    torch.cuda.synchronize()
    want = rank.results()
    for k in range(40):
        rank.call()
        if k % 2:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert _same(rank.results(), want)
    assert ddp.ddp_device_status() == 0


TIMEOUT = -4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("grads,tile", [(False, 0), (False, 11), (True, 5)])
def test_a_products_wait_that_runs_out_ends_the_call(dtype, grads, tile):
    """A planted stall: the loads of one block stop before a tile, as if it never came.  Nothing is in flight then and every
    wait has its limit, 2 s for these kernels, so the call ends, says so, and the next one gives its bits again."""
    rank = Rank([300, 200], 3000, 192, dtype, 9)          # 2 to 3 tiles of rows by 12 of columns

    def call():
        if grads:
            rank.call()
            return rank.results()
        return [rank.head.cross_entropy(rank.hidden, rank.targets).clone()]

    ddp.ddp_device_status(clear=True)
    want = call()
    torch.cuda.synchronize()
    limit = ddp.ddp_set_wait_limit_ms(100)
    try:
        ddp.ddp_plant_stall(tile)
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        ddp.ddp_plant_stall(-1)
        ddp.ddp_set_wait_limit_ms(limit)
    assert ddp.ddp_device_status(clear=True) == TIMEOUT
    assert 1.9 <= dt < 8.0, dt
    for _ in range(2):
        assert _same(call(), want)
    torch.cuda.synchronize()
    assert ddp.ddp_device_status() == 0


def test_a_plant_beyond_the_products_tiles_stalls_nothing():
    rank = Rank([300, 200], 3000, 192, torch.bfloat16, 9)
    want = rank.head.cross_entropy(rank.hidden, rank.targets).clone()
    for _ in range(2):
        ddp.ddp_plant_stall(1 << 40)
        got = rank.head.cross_entropy(rank.hidden, rank.targets)
        torch.cuda.synchronize()
        assert ddp.ddp_device_status() == 0 and torch.equal(got, want)
    ddp.ddp_plant_stall(-1)
