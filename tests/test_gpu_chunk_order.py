"""GPU tests of requests with many rows whose runs of one and of two row tiles share a block: short contexts,
so that most runs have one key tile and the roles are as far apart as they get, in few blocks, many times."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from chunk_util import PAGE, ChunkCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def lengths(kinds, n, rng):
    """n requests of the kinds in turn, "1" (17 to 128 rows) or "2" (more), with g = 8 query heads a kv head:
    one key tile each, now and then two or three."""
    seq, new = [], []
    for b in range(n):
        new.append(int(rng.integers(3, 17) if kinds[b % len(kinds)] == "1" else rng.integers(17, 61)))
        seq.append(int(rng.integers(0, 128 - new[-1] + 1) if rng.random() < 0.8 else rng.integers(130, 330)))
    return seq, new


@pytest.mark.parametrize("d,masked", [(64, True), (128, False)])
@pytest.mark.parametrize("n_sms,kinds", [(1, "12"), (2, "12"), (3, "112"), (7, "1222"), (2, "11112"), (152, "12")])
def test_runs_of_one_key_tile_take_turns(d, masked, n_sms, kinds):
    rng = np.random.default_rng(1000 * n_sms + len(kinds))
    seq, new = lengths(kinds, 40 if n_sms < 100 else 400, rng)
    c = ChunkCase(seq, new, hq=16, hkv=2, d=d, seed=n_sms)
    if masked:
        c.excl = np.zeros((c.n, c.max_pages), dtype=np.uint16)
        for b in range(c.n):
            for j in range(c.seq[b]):
                if rng.random() < 0.2:
                    c.excl[b, j // PAGE] |= np.uint16(1 << (j % PAGE))
    c.to_device()
    c.L.dims.n_sms = n_sms
    got = c.step()
    first = c.out.clone()
    for _ in range(20):
        c.out.fill_(3.0)
        c.attend()
        pcf.check_device_error()
        assert torch.equal(c.out, first)
    c.check(got)
