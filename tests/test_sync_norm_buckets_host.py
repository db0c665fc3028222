"""Where a sync with norm may put its norms, with the algorithms that use bucket buffers.

Every call here is refused by the host checks, so no made-up pointer reaches the GPU.
"""
import ctypes

import pytest

import gradient_sync_plan_gb300 as ddp

H = 0x7f0000000000                     # made-up device addresses, never dereferenced
WS = H + (1 << 40)


def _create(algo, buckets, bucket_numel, world=2):
    """world ranks with a member of 8 elements in each bucket."""
    n = len(bucket_numel)
    vp = lambda p: (ctypes.c_void_p * len(p))(*p)
    i64 = lambda v: (ctypes.c_int64 * len(v))(*v)
    h = ctypes.c_void_p()
    st = ddp.lib().ddp_sync_norm_create(world, n, vp([H + (k << 12) for k in range(world * n)]), i64([8] * n),
                                        (ctypes.c_int32 * n)(*range(n)), i64([0] * n), n, i64(bucket_numel), vp(buckets),
                                        ddp.F32, world, algo, WS, 1 << 20, ctypes.byref(h))
    assert st == 0
    return h


@pytest.mark.parametrize("algo,size", [(ddp.DDP_ALGO_FUSED, 4), (ddp.DDP_ALGO_STAGED, 4), (ddp.DDP_ALGO_BF16_HOOK, 2)])
def test_norms_inside_a_bucket_are_refused(algo, size):
    # rank 0's and rank 1's buffers of two buckets; the second ones share memory with the first and reach past them
    first, second = H + (1 << 30), H + (2 << 30)
    h = _create(algo, [first, first + 16 * size, second, second + 16 * size], [64, 64])
    run = ddp.lib().ddp_sync_norm_run
    end = (16 + 64) * size
    for base in (first, second):
        for norms in (base - 4, base, base + 8, base + 64 * size - 4, base + 64 * size, base + end - 4):
            assert run(h, norms, None) == -1, (norms - base)
    ddp.lib().ddp_sync_norm_destroy(h)


def test_norms_between_buckets_that_overlap_each_other():
    """A long bucket that starts first and a short one inside it: what lies behind the short one is still the long one's."""
    a = H + (1 << 30)
    h = _create(ddp.DDP_ALGO_FUSED, [a, a + 64, a + (1 << 20), a + (1 << 20) + 64], [256, 8])
    run = ddp.lib().ddp_sync_norm_run
    for at in (a + 200, a + 512, a + 1020, a + (1 << 20) + 900):
        assert run(h, at, None) == -1
    ddp.lib().ddp_sync_norm_destroy(h)
