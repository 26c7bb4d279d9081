"""GPU tests of trees whose runs of one and of two row tiles share a block: short contexts, so that most runs have a
unit or two and the roles are as far apart as they get, in few blocks, many times."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from tree_util import TreeCase, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def batch(kinds, n, rng):
    """n requests of the kinds in turn, "1" (up to 128 rows), "2" (up to 256) or "3" (more, its last pair of either
    kind), with g = 8 query heads a kv head: a unit each, now and then several."""
    top = {"1": 17, "2": 33, "3": 80}
    low = {"1": 1, "2": 17, "3": 33}
    seq, parents = [], []
    for b in range(n):
        k = kinds[b % len(kinds)]
        m = int(rng.integers(low[k], top[k]))
        parents.append(random_tree(m, rng, 6))
        seq.append(int(rng.integers(0, 30)) if rng.random() < 0.7 else int(rng.integers(60, 400)))
    return seq, parents


@pytest.mark.parametrize("d,masked", [(64, True), (128, False), (128, True)])
@pytest.mark.parametrize("n_sms,kinds", [(1, "12"), (2, "1"), (3, "112"), (7, "123"), (2, "11112"), (152, "123")])
def test_short_runs_take_turns(d, masked, n_sms, kinds):
    rng = np.random.default_rng(100 * n_sms + len(kinds))
    seq, parents = batch(kinds, 30 if n_sms < 100 else 200, rng)
    c = TreeCase(seq, parents, hq=16, hkv=2, d=d, seed=n_sms)
    if masked:
        c.excl = np.zeros((c.n, c.max_pages), dtype=np.uint16)
        for b in range(c.n):
            for j in range(c.seq[b]):
                if rng.random() < 0.2:
                    c.excl[b, j // 16] |= np.uint16(1 << (j % 16))
    c.to_device()
    c.L.dims.n_sms = n_sms
    got = c.step()
    first = c.out.clone()
    for _ in range(20):
        c.out.fill_(3.0)
        c.ws.fill_(255)
        c.attend()
        pcf.check_device_error()
        assert torch.equal(c.out, first)
    c.check(got, rows=10)


@pytest.mark.parametrize("sizes", [[200], [256, 3]])
def test_as_many_row_pairs_as_nodes_allow(sizes):
    """128 query heads on one kv head: two nodes a row pair."""
    rng = np.random.default_rng(3)
    c = TreeCase([70, 5][: len(sizes)], [random_tree(n, rng, 20) for n in sizes], hq=128, hkv=1, d=64).to_device()
    c.check(c.step(), rows=6)
