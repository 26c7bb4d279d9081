"""GPU tests of the tree attention with very large values: a weighted mean of finite values is finite, and so is what
the kernel sums up on the way to it, as long as |v| stays below 2^112 (or slots * |v| below 2^132)."""
from __future__ import annotations

import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from tree_scores import UNIT, leveled, moves_once, pair

pytestmark = pytest.mark.gpu

RANGE = -8


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def scaled(c, by):
    for t in (c.v_pool, c.v_new):
        t.copy_((t.float().clamp(-3.0, 3.0) * by).to(torch.bfloat16))
    return c.to_device()


# In a context of n slots the sums stay below ceil(n / 32) |v| (1 + 2^-8): 3 * 2^120 * 16 = 2^125.6 here.
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [16, 50])
@pytest.mark.parametrize("n_sms", [1, 3])
@pytest.mark.parametrize("power", [110, 115, 120])
def test_weights_far_above_the_first_ones_meet_large_values(power, n_sms, nodes, d):
    """The weights of 2^14.9 against the first scores, below what moves a reference."""
    c = scaled(leveled([moves_once(5, 1), dict(slots=300, at=pair(40, 14.9))], [nodes, nodes], d=d, seed=power), 2.0 ** power)
    c.L.dims.n_sms = n_sms
    c.check(c.step(), rows=8)


@pytest.mark.parametrize("nodes", [16, 50])
def test_the_largest_value_of_any_context(nodes):
    """Every half unit holds such a weight: the sums come as near their limit as they can."""
    at = {}
    for h in range(1, 128):
        at.update(pair(32 * h + (5 * h) % 30, 14.9))
    c = scaled(leveled([dict(slots=64 * UNIT, at=at)], [nodes], d=128, seed=2), 2.0 ** 110)
    c.L.dims.n_sms = 1
    c.check(c.step(), rows=8)


@pytest.mark.parametrize("n_sms", [1, 3])
def test_values_as_large_as_bf16_holds_in_a_short_context(n_sms):
    c = leveled([dict(slots=60, at={}), dict(slots=200, at={})], [7, 33], d=128, seed=5)
    for t in (c.v_pool, c.v_new):
        t.copy_(torch.where(t > 0, 1.0, -1.0) * 3.3e38)
    c.to_device()
    c.L.dims.n_sms = n_sms
    c.check(c.step(), rows=8)


def test_a_value_that_is_not_finite_is_still_reported():
    for value in (float("inf"), float("nan")):
        c = leveled([moves_once(3, 0)], [20], d=128)
        c.v_pool[c.bt[0, 2], 1, 3, 9] = value
        c.to_device()
        c.tables()
        c.append()
        c.attend()
        with pytest.raises(pcf.PcfError) as e:
            pcf.check_device_error()
        assert e.value.status == RANGE
