"""GPU tests of long contexts with checks that see a lost or doubled page: keys planted at the borders of the
work's shares, of key tiles and of the context, and the norm of every row's error."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from chunk_long import PAGE, outside, plant
from chunk_util import ChunkCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def share_borders(c, b):
    """Pages on both sides of where shares of request b's work begin, in the words of the plan (its layout:
    chunk_format.h): {request, kv head, page, ..} a worker of the few-row kernel, {request, kv head, row pair,
    key tile; ..} a block of the other one."""
    plan = c.L.plan.cpu().numpy()
    blocks = c.L.dims.n_sms
    workers = 12 * blocks
    at = (4 + 9 * (c.n + 1) + 3) // 4 * 4
    few = plan[at: at + 12 * workers].reshape(workers, 12)
    many = plan[at + 12 * (workers + 1):][: 8 * blocks].reshape(blocks, 8)
    pages = {int(p) for r, _, p in few[:, :3] if r == b} | {8 * int(w[3]) for w in many if w[0] == b and w[4] > 0}
    return sorted({x for p in pages for x in (p - 1, p) if x >= 0})


@pytest.mark.parametrize("seq,new,shape", [
    ([9000], [1], dict(hq=32, hkv=8, d=128)), ([33000], [1], dict(hq=32, hkv=8, d=128)),
    ([9000, 17, 2500], [1, 1, 3], dict(hq=32, hkv=8, d=128)), ([16000], [2], dict(hq=8, hkv=2, d=64)),
    ([5000] * 3, [4, 1, 2], dict(hq=16, hkv=4, d=128)),
    ([9000], [20], dict(hq=32, hkv=8, d=128)), ([33000], [33], dict(hq=8, hkv=2, d=64)),
    ([9000], [200], dict(hq=32, hkv=8, d=128)), ([33000], [70], dict(hq=16, hkv=4, d=128)),
    ([6000, 9000, 4000, 300], [150, 30, 1, 400], dict(hq=32, hkv=8, d=64))])
@pytest.mark.parametrize("n_sms", [None, 3])
def test_no_page_is_lost_or_counted_twice(seq, new, shape, n_sms):
    c = ChunkCase(seq, new, seed=sum(seq), stale="normal", **shape).to_device()
    if n_sms is not None:
        c.L.dims.n_sms = n_sms
    c.tables()
    pcf.check_device_error()
    rng = np.random.default_rng(sum(new))
    rows = []
    for b in range(c.n):
        n = c.seq[b] + c.new[b]
        some = sorted({0, c.new[b] - 1, *rng.integers(0, c.new[b], 3)})
        borders = share_borders(c, b)
        rng.shuffle(borders)
        plant(c, b, [0, c.seq[b] // PAGE - 1, c.seq[b] // PAGE, 7, 8] + borders[: 40] + rng.integers(0, n // PAGE, 8).tolist(),
              some)
        rows.append(some)
    for dev, host in ((c.dk, c.k_pool), (c.dv, c.v_pool), (c.dkn, c.k_new), (c.dvn, c.v_new)):
        dev.copy_(host)
    c.append()
    c.attend()
    pcf.check_device_error()
    got = c.out.float().cpu().double().numpy()
    for b in range(c.n):
        t, exact = c.oracle(b, rows[b])
        wrong = outside(got[c.base[b] + t], *exact)
        assert wrong is None, (b, c.seq[b], c.new[b], wrong)
    first = c.out.clone()
    c.attend()
    pcf.check_device_error()
    assert torch.equal(c.out, first)
