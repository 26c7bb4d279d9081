"""CPU tests that the checks of long contexts see what they are for: the oracle with a page lost, doubled or
exchanged is rejected, wherever the page is, and a result rounded like the kernels' is not."""
import numpy as np
import pytest

from oracle import chunk

from chunk_long import PAGE, outside, plant
from chunk_util import ChunkCase


def to_bf16(x):
    """Rounded to 8 bits of mantissa, to the nearest."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 256) / 256, e)


def context(n, new, seed, pages=None, d=128, hq=4, hkv=2):
    """One request of n tokens with `new` more; returns (attend(changed keys) -> results, its exact results)."""
    c = ChunkCase([n], [new], hq=hq, hkv=hkv, d=d, seed=seed, stale="normal", max_chunk=new)
    rows = [0, new - 1] if new > 1 else [0]
    if pages is not None:
        plant(c, 0, pages, rows)
    total = n + new
    k, v = c.k_pool.double().numpy().copy(), c.v_pool.double().numpy().copy()
    k[c.slots // PAGE, :, c.slots % PAGE] = c.k_new.double().numpy()
    v[c.slots // PAGE, :, c.slots % PAGE] = c.v_new.double().numpy()
    table = c.bt[0, : -(-total // PAGE)]
    K, V = chunk.gather(k, table, total), chunk.gather(v, table, total)
    pos = (c.pp[0, : len(table), None] + np.arange(PAGE)).reshape(-1)[:total]
    t = np.array(rows)
    seen = np.arange(total)[None] <= n + t[:, None]

    def attend(order=None):
        """The slots of `order` in the place of all of them."""
        o = np.arange(total) if order is None else order
        return chunk.attention(c.q.double().numpy()[t], c.where[t], K[o], V[o], pos[o], seen[:, o], c.theta)

    return c, attend


@pytest.mark.parametrize("n,new,d", [(9000, 1, 128), (9000, 40, 64), (33000, 1, 128)])
def test_a_page_lost_or_doubled_or_exchanged_is_seen(n, new, d):
    c, attend = context(n, new, seed=n + d, d=d)
    exact = attend()
    assert outside(to_bf16(exact[0]), *exact) is None
    slots = np.arange(n + new)
    last = (n + 1) // PAGE - 1                       # the last page that the first row sees whole
    for p in (0, 1, last // 3, last // 2, last):
        mine = slots // PAGE == p
        for what, order in (("lost", slots[~mine]), ("doubled", np.concatenate([slots, slots[mine]]))):
            assert outside(attend(order)[0], *exact), (what, p)
        other = slots.copy()
        other[mine] = slots[slots // PAGE == (p + 5) % last]
        assert outside(attend(other)[0], *exact), ("exchanged", p)


@pytest.mark.parametrize("n,new,d", [(9000, 1, 128), (9000, 40, 64), (33000, 1, 128)])
def test_a_planted_page_lost_or_doubled_leaves_the_elementwise_bound(n, new, d):
    total = n + new
    pages = [0, 7, 8, n // 32, (n + 1) // PAGE - 1, n // PAGE]
    c, attend = context(n, new, seed=n + d + 1, pages=pages, d=d, hq=8)
    exact = attend()
    assert outside(to_bf16(exact[0]), *exact) is None
    lim = chunk.attention_bound(*exact)
    slots = np.arange(total)
    used = sorted({(j // PAGE) for j in range(total) if np.any(np.abs(
        (c.v_new[j - n] if j >= n else c.v_pool[c.bt[0, j // PAGE], :, j % PAGE]).double().numpy()).min(axis=-1) == 4.0)})
    assert set(pages) - {n // PAGE} <= set(used)
    for p in used:
        mine = slots // PAGE == p
        for what, order in (("lost", slots[~mine]), ("doubled", np.concatenate([slots, slots[mine]]))):
            assert (np.abs(attend(order)[0] - exact[0]) > lim).any(), (what, p)
