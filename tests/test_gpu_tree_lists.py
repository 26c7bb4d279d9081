"""GPU tests of what tree_accept leaves of the free list where it refuses to give pages back."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from chunk_util import PAGE
from tree_util import TreeCase, random_tree, star

pytestmark = pytest.mark.gpu

BOUNDS = -6


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def raises(status):
    with pytest.raises(pcf.PcfError) as e:
        pcf.check_device_error()
    assert e.value.status == status


def in_use(c, length):
    return [p for b in range(c.n) for p in c.L.block_table[b, : -(-length[b] // PAGE)].tolist()]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("short", [1, 2, 5])
def test_a_refused_list_keeps_its_head(in_place, short):
    """Two requests whose branches each need one of the pages they took: the list's next entry is the first one's second
    page, the entry behind the second one's first, which it still holds."""
    c = TreeCase([16, 32], [star(40), star(40)], max_pages=8).to_device()
    c.choice[:] = -5                                # (only the first node of each, which is certain, is kept)
    c.d_choice.fill_(-5)
    if in_place:
        c.d_seq_out, c.d_head_out = c.d_seq, c.d_head
    c.tables()
    pcf.check_device_error()
    whole = c.d_free.clone()
    c.d_free = whole[: c.head - short].clone()
    before = c.d_free.clone()
    c.accept()
    raises(BOUNDS)
    assert torch.equal(c.d_free, before) and c.d_head_out.item() == c.head
    length = c.d_seq_out.tolist()
    assert length == [17, 33]
    # no page that the branches hold is behind the head
    assert not set(in_use(c, length)) & set(whole[c.d_head_out.item():].tolist())
    # the right list mends it
    c.d_free = whole
    c.accept()
    pcf.check_device_error()
    path, kept, token, length, free, head = c.accepted()
    assert c.d_seq_out.tolist() == length and c.d_head_out.item() == head and c.d_free.tolist() == [int(x) for x in free]


def test_steps_behind_a_refused_list_share_no_page():
    c = TreeCase([14, 3, 40], [random_tree(n, np.random.default_rng(n), 4) for n in (40, 33, 64)], vocab=2,
                 extra_pages=40, max_pages=12).to_device()
    c.d_seq_out, c.d_head_out = c.d_seq, c.d_head
    c.tables()
    whole = c.d_free
    c.d_free = whole[:2].clone()
    c.accept()
    raises(BOUNDS)
    c.d_free = whole
    c.d_next = None
    for _ in range(3):                              # (on with the real list)
        c.tables()
        c.accept()
        pcf.check_device_error()
        used = in_use(c, c.d_seq.tolist())
        free = whole[c.d_head.item():].tolist()
        assert len(set(used)) == len(used) and not set(used) & set(free)
