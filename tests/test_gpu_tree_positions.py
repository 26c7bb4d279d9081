"""GPU tests of trees near the end of the cos/sin table: it must reach as far as a line of all the nodes would, to the
end of its last page."""
from __future__ import annotations

import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from chunk_util import PAGE
from tree_util import TreeCase, star

pytestmark = pytest.mark.gpu

BOUNDS = -6


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


# (page p's first position is 5 + 16 p: a table of `pages` pages ends at 5 + 16 pages)
@pytest.mark.parametrize("seq,nodes,pages", [(20, 40, 4), (32, 16, 3), (0, 128, 8), (31, 1, 2)])
def test_the_table_reaches_to_the_end_of_the_last_node_s_page(seq, nodes, pages):
    for short in (0, 1):
        c = TreeCase([seq], [star(nodes)])             # (two positions deep at most)
        c.max_pos = 5 + PAGE * pages - short
        c.to_device()
        if not short:
            c.check(c.step(), rows=6)
            continue
        c.tables()
        with pytest.raises(pcf.PcfError) as e:
            pcf.check_device_error()
        assert e.value.status == BOUNDS
        c.append()
        c.attend()
        pcf.check_device_error()
        assert bool((c.tree.row_pos == -1).all()) and bool((c.out == 3.0).all()) and c.d_seq_out.tolist() == [seq]


def test_fewer_nodes_fit():
    """The same request with the nodes that the table has room for."""
    c = TreeCase([20], [star(28)])
    c.max_pos = 5 + PAGE * 3
    c.check(c.to_device().step(), rows=6)
