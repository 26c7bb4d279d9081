"""GPU tests of the order of a step's calls: trees that are not of the last chunk are not accepted."""
from __future__ import annotations

import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from tree_util import TreeCase, chain, star

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


def case():
    return TreeCase([14, 30], [chain(20), star(12)], vocab=1, extra_pages=30, max_pages=12, stale="normal").to_device()


def check_accepted(c):
    path, kept, token, length, free, head = c.accepted()
    assert c.tree.path.tolist() == path and c.tree.n_kept.tolist() == kept and c.tree.next_token.tolist() == token
    assert c.d_seq_out.tolist() == length and c.d_head_out.item() == head and c.d_free.tolist() == [int(x) for x in free]


@pytest.mark.parametrize("in_place", [False, True])
def test_trees_of_an_earlier_chunk_are_not_accepted(in_place):
    c = case()
    if in_place:
        c.d_seq_out, c.d_head_out = c.d_seq, c.d_head
        c.d_next = None
    c.tables()
    c.append()
    c.accept()
    pcf.check_device_error()
    super(TreeCase, c).tables()                         # the next chunk without its trees
    pcf.check_device_error()
    after = [t.clone() for t in (c.tree.path, c.tree.next_token, c.d_seq_out, c.d_head_out, c.d_free, c.dk, c.dv)]
    c.accept()
    raises(BOUNDS)
    assert c.tree.n_kept.tolist() == [0, 0]
    pcf.tree_keep(c.L, c.tree, [c.dk], [c.dv])          # moves nothing
    pcf.check_device_error()
    for old, new in zip(after, (c.tree.path, c.tree.next_token, c.d_seq_out, c.d_head_out, c.d_free, c.dk, c.dv)):
        assert torch.equal(old, new)
    pcf.tree_tables(c.L, c.tree, c.d_parent)            # with them it goes on
    c.accept()
    pcf.check_device_error()
    assert c.tree.n_kept.tolist() == [20, 2]            # (of siblings with the chosen token the first)


def test_more_than_one_tree_on_a_chunk():
    """Two candidates for the same rows: each DraftTree is of the last chunk."""
    c = case()
    c.tables()
    other = pcf.DraftTree(c.L)
    pcf.tree_tables(c.L, other, c.d_parent)
    c.accept()
    pcf.check_device_error()
    check_accepted(c)
    c.tree = other
    c.accept()
    pcf.check_device_error()
    check_accepted(c)


def test_a_plan_may_hold_anything_before():
    c = case()
    c.L.plan.fill_(-1)
    c.tree.plan.fill_(2 ** 31 - 1)
    for _ in range(3):
        c.tables()
        c.accept()
        pcf.check_device_error()
        check_accepted(c)


def test_replayed_steps_are_each_their_own():
    c = case()
    c.tables(), c.accept()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.tables()
        c.accept()
    for _ in range(5):
        graph.replay()
        pcf.check_device_error()
        check_accepted(c)
