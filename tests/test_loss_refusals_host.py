"""Temperatures that binary32 cannot compute with are refused before any launch; the others next to them are not."""
import pytest

import gradient_sync_plan_gb300 as ddp
from test_loss_head_host import LOSS, _args, _call, _create


@pytest.mark.parametrize("fn", ["ddp_distill", "ddp_distill_grad"])
# 1.5 / 4e-39 and (1e20)^2 are beyond binary32's 3.4e38
@pytest.mark.parametrize("temperature", [4e-39, 3e-39, 1e20, 3e38])
def test_temperatures_beyond_the_arithmetic(fn, temperature):
    st, h = _create()
    assert st == 0
    assert _call(h, fn, _args(temperature=temperature)) == -1
    ddp.lib().ddp_loss_head_destroy(h)


@pytest.mark.parametrize("temperature", [1e-38, 0.01, 1.0, 1e4, 1.8e19])
def test_temperatures_that_are_taken_reach_the_next_check(temperature):
    st, h = _create()
    assert st == 0
    assert _call(h, "ddp_distill", _args(temperature=temperature, loss=LOSS + 2)) == -2       # an unaligned loss
    ddp.lib().ddp_loss_head_destroy(h)
