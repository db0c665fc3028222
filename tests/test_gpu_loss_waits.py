"""Calls of the loss head that follow each other closely: every one ends, and repeats its bits."""
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
