"""Float32 sums from the tensor cores, on average over many: what their cutting of low bits takes off is put back.

The tensor cores cut a long sum's low bits a step of 16 products, by 1.6e-8 of the result on average.  Logits and float32
gradients are scaled back by that; each test asks that what is left is less than half of it, over so many sums that their
own roundings average out.
"""
import pytest
import torch

import gradient_sync_plan_gb300 as ddp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
CUT = 1.6e-8                           # a step of 16 products
TYPES = pytest.mark.parametrize("dtype", [BF16, F32])


def _bias(got, want):
    """The part of `got - want` that is a multiple of `want`."""
    return float(((got.double() - want) * want).sum() / (want * want).sum())


@TYPES
@pytest.mark.parametrize("dim,tokens", [(1024, 4096), (4096, 4096), (16384, 2048), (65536, 512)])
def test_logits_are_not_small_on_average(dim, tokens, dtype):
    # two columns of which the target's weights are 0: with the other logit above 16 the loss is that logit, to 2^-23 of it.
    # 2^-24 of rounding each, over 512 losses at least, is 2.7e-9 on average; the cut is 1e-6 to 6.6e-5
    gen = torch.Generator(device="cuda").manual_seed(dim)
    kw = dict(device="cuda", generator=gen)
    w = torch.stack([torch.zeros(dim, device="cuda"), torch.randn(dim, **kw) * dim ** -0.5]).to(dtype)
    h = (torch.randn(tokens, dim, **kw) + (22.0 + 10.0 * torch.rand(tokens, 1, **kw)) * w[1].float()).to(dtype)
    losses = torch.empty(tokens, device="cuda")
    ddp.LossHead([w], max_tokens=tokens).cross_entropy([h], [torch.zeros(tokens, dtype=torch.int64, device="cuda")],
                                                       token_losses=[losses])
    torch.cuda.synchronize()
    z = h.double() @ w[1].double()
    assert float(z.min()) > 16
    assert abs(_bias(losses, z + torch.log1p(torch.exp(-z)))) < 0.5 * CUT * dim / 16


@TYPES
def test_a_small_correction_is_no_larger_than_it_is(dtype):
    # logits that are exact, over a depth whose correction, 6.4e-8, is no multiple of a float's step from 1: they may come
    # out larger by it and half of it, not by 1.2e-7
    tokens, dim = 2000, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = torch.zeros(2, dim, device="cuda")
    w[1] = (32.0 + 31.0 * torch.rand(dim, device="cuda", generator=gen)).bfloat16().float()
    h = torch.eye(dim, device="cuda").repeat(tokens // dim + 1, 1)[:tokens]
    losses = torch.empty(tokens, device="cuda")
    ddp.LossHead([w.to(dtype)], max_tokens=tokens).cross_entropy([h.to(dtype)], [torch.zeros(tokens, dtype=torch.int64, device="cuda")],
                                                                 token_losses=[losses])
    torch.cuda.synchronize()
    assert abs(_bias(losses, h.double() @ w[1].double())) < 1.5 * CUT * dim / 16


@pytest.mark.parametrize("tokens,vocab,dim", [(1024, 50257, 512), (2000, 20000, 1024), (1500, 2048, 256)])
def test_float32_gradients_are_not_small_on_average(tokens, vocab, dim):
    # of 1024 of the depth (or all of it) a part: 1e-6; an element's own error, some 1e-6 of the mean, over 1e5 elements
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    kw = dict(device="cuda", generator=gen)
    w, h = torch.randn(vocab, dim, **kw) * dim ** -0.5, torch.randn(tokens, dim, **kw)
    y = torch.randint(0, vocab, (tokens,), **kw)
    gw, gh = torch.empty_like(w), torch.empty_like(h)
    ddp.LossHead([w], [gw], max_tokens=tokens).cross_entropy_grad([h], [y], [gh], reduction=ddp.DDP_LOSS_SUM)
    torch.cuda.synchronize()
    dz = torch.softmax(h.double() @ w.double().t(), 1)
    dz[torch.arange(tokens, device="cuda"), y] -= 1
    assert abs(_bias(gh, dz @ w.double())) < 0.5 * CUT * min(vocab, 1024) / 16
    assert abs(_bias(gw, dz.t() @ h.double())) < 0.5 * CUT * min(tokens, 1024) / 16
