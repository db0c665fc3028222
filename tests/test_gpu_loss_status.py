"""The device status word where a wait that ran out and a column outside the vocabulary meet: the wait is what counts."""
import pytest
import torch

import gradient_sync_plan_gb300 as ddp
import workloads

pytestmark = pytest.mark.gpu
INVALID, TIMEOUT = -1, -4


def _time_out():
    """A fused ring whose one producer stops before a tile (ddp_plant_stall), so that its consumers' wait runs out."""
    limit, kernel = ddp.ddp_set_wait_limit_ms(100), ddp.ddp_set_fused_kernel(ddp.DDP_FUSED_TMA)
    try:
        x = workloads.rank_vectors(8, 1 << 21, "randn", std=1e-2, seed0=51).cuda()
        ddp.ddp_plant_stall(3)
        ddp.ring_allreduce_fused(x, 8)
        torch.cuda.synchronize()
    finally:
        ddp.ddp_plant_stall(-1)
        ddp.ddp_set_fused_kernel(kernel)
        ddp.ddp_set_wait_limit_ms(limit)


def _bad_column(tokens, vocab, dim, distill):
    """A loss with one target, or one teacher's index, that is no column."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    kw = dict(device="cuda", generator=gen)
    w, h = torch.randn(vocab, dim, **kw), torch.randn(tokens, dim, **kw)
    y = torch.randint(0, vocab, (tokens,), **kw)
    head = ddp.LossHead([w], max_tokens=tokens, max_teacher=2)
    if distill:
        indices = torch.randint(0, vocab, (tokens, 2), **kw)
        indices[1, 1] = vocab
        head.distill([h], [torch.randn(tokens, 2, **kw)], [indices])
    else:
        y[1] = vocab
        head.cross_entropy([h], [y])
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens,vocab,dim", [(7, 100, 32), (130, 777, 128)])     # one launch; the tensor cores' kernels
@pytest.mark.parametrize("distill", [False, True])
def test_a_wait_that_ran_out_outlasts_a_bad_column(tokens, vocab, dim, distill):
    ddp.ddp_device_status(clear=True)
    _bad_column(tokens, vocab, dim, distill)
    assert ddp.ddp_device_status(clear=False) == INVALID
    _bad_column(tokens, vocab, dim, distill)
    assert ddp.ddp_device_status(clear=False) == INVALID
    _time_out()
    assert ddp.ddp_device_status(clear=False) == TIMEOUT
    _bad_column(tokens, vocab, dim, distill)
    assert ddp.ddp_device_status(clear=True) == TIMEOUT
    _bad_column(tokens, vocab, dim, distill)
    assert ddp.ddp_device_status(clear=True) == INVALID and ddp.ddp_device_status() == 0
