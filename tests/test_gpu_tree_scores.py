"""GPU tests of the tree attention where scores grow along a request, so that rows' references move behind their
first unit and what they have summed up is scaled down: in either half of a unit, in both, in units one behind the
other, in runs of one and of two row tiles, in one block and across blocks.  (tests/test_tree_scores_host.py shows
on the CPU that these requests do that, and that a result left as it was leaves the bound.)"""
from __future__ import annotations

import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from tree_scores import UNIT, both_halves, leveled, moves_once, pair

pytestmark = pytest.mark.gpu

SHAPES = [dict(hq=8, hkv=2, d=64), dict(hq=8, hkv=2, d=128), dict(hq=16, hkv=2, d=128)]
IDS = ["8-2-64", "8-2-128", "16-2-128"]


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def check(c, n_sms):
    c.to_device()
    if n_sms is not None:
        c.L.dims.n_sms = n_sms
    got = c.step()
    first = c.out.clone()
    for _ in range(3):
        c.out.fill_(3.0)
        c.ws.fill_(255)
        c.attend()
        pcf.check_device_error()
        assert torch.equal(c.out, first)
    c.check(got, rows=8)


@pytest.mark.parametrize("n_sms", [1, 3])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("nodes", [16, 50, 100])               # one row tile, two, more than one pair
@pytest.mark.parametrize("unit", [1, 2, 3, 5])
def test_a_reference_moves(unit, nodes, shape, n_sms):
    check(leveled([moves_once(unit, 0), moves_once(unit, 1), both_halves(unit)], [nodes, nodes, nodes], seed=unit, **shape),
          n_sms)


@pytest.mark.parametrize("n_sms", [1, 2])
@pytest.mark.parametrize("shape", SHAPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("nodes", [16, 50])
@pytest.mark.parametrize("first,second", [((1, 0), (1, 1)), ((2, 0), (2, 1)), ((2, 1), (3, 0)), ((2, 1), (4, 0)), ((1, 1), (3, 1)),
                                          ((2, 0), (5, 1))])
def test_a_reference_moves_twice(first, second, nodes, shape, n_sms):
    check(leveled([moves_once(*first, second), moves_once(2, 1)], [nodes, nodes], seed=7, **shape), n_sms)


@pytest.mark.parametrize("n_sms", [2, 5, 14])
@pytest.mark.parametrize("shape", SHAPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("nodes", [16, 50])
@pytest.mark.parametrize("rising", [True, False])
def test_parts_whose_references_differ(rising, nodes, shape, n_sms):
    """A level every unit, 5 bits apart: each part has another reference, and the parts' sums meet in the join."""
    units = 14
    at = {}
    for u in range(units):
        at.update(pair(UNIT * u + (11 * u) % 60, 5.0 * (u if rising else units - 1 - u) - 20.0))
    check(leveled([dict(slots=UNIT * units, at=at)], [nodes], seed=3, **shape), n_sms)
