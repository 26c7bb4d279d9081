"""GPU tests of what the tables and append calls refuse on the device, whole or row by row."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf

from chunk_util import PAGE, ChunkCase

pytestmark = pytest.mark.gpu

BOUNDS = -6


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def refused():
    with pytest.raises(pcf.PcfError) as e:
        pcf.check_device_error()
    assert e.value.status == BOUNDS


# seq 26, 32, 0: a started page, a full one, none
STARTED = {
    "started page before position 0": lambda c: (c.L.page_pos.__setitem__((0, 1), -5), c.d_next.__setitem__(0, 5)),
    "started page at -16": lambda c: (c.L.page_pos.__setitem__((0, 1), -16), c.d_next.__setitem__(0, -6)),
    "started page behind the pool": lambda c: c.L.block_table.__setitem__((0, 1), c.n_phys),
    "started page without a number": lambda c: c.L.block_table.__setitem__((0, 1), -1),
}
# (with next_pos nothing is read of a full page)
FULL = {"full page before position 0": lambda c: c.L.page_pos.__setitem__((1, 1), -5)}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("what,next_pos", [(w, n) for w in STARTED for n in (True, False)] + [(w, False) for w in FULL])
def test_bad_entries_of_pages_held_refuse_the_whole_call(what, next_pos, in_place):
    c = ChunkCase([26, 32, 0], [3, 5, 17], max_pages=6, max_chunk=20, stale="normal").to_device()
    {**STARTED, **FULL}[what](c)
    if not next_pos:
        c.d_next = None
    if in_place:
        c.d_seq_out, c.d_head_out = c.d_seq, c.d_head
    seq, head = c.d_seq.clone(), c.d_head.clone()
    table, pos, k = c.L.block_table.clone(), c.L.page_pos.clone(), c.dk.clone()
    c.tables()
    c.append()
    refused()
    assert torch.equal(c.L.block_table, table) and torch.equal(c.L.page_pos, pos)
    assert torch.equal(c.d_seq_out, seq) and torch.equal(c.d_head_out, head)
    assert bool((c.L.slot_map == -1).all()) and bool((c.L.row_pos == -1).all()) and not bool(c.L.row_base.any())
    assert torch.equal(c.dk, k)


def test_idle_requests_and_full_pages_with_next_pos_may_hold_what_they_like():
    """What a call does not read it does not refuse."""
    c = ChunkCase([26, 32, 20], [0, 5, 1], max_pages=6, stale="normal").to_device()
    c.L.page_pos[0, 1], c.L.block_table[0, 1] = -5, -1
    c.L.page_pos[1, 1], c.L.block_table[1, 1] = -5, -1
    c.tables()
    pcf.check_device_error()
    assert np.array_equal(c.L.slot_map.cpu().numpy(), c.slots) and np.array_equal(c.L.row_pos.cpu().numpy(), c.where)


def test_rows_of_a_layout_without_tables_go_nowhere():
    c = ChunkCase([20], [4], stale="normal").to_device()
    k, v = c.dk.clone(), c.dv.clone()
    c.append()
    pcf.check_device_error()
    assert torch.equal(c.dk, k) and torch.equal(c.dv, v)


@pytest.mark.parametrize("row_pos", [False, True])
@pytest.mark.parametrize("slot", [-2, -2 ** 31, "end", 2 ** 31 - 1])
def test_append_reports_slots_outside_the_pool(slot, row_pos):
    c = ChunkCase([20, 7], [4, 9], stale="normal").to_device()
    c.tables()
    c.L.slot_map[2] = c.n_phys * PAGE if slot == "end" else slot
    k, page, r = c.dk.clone(), c.slots // PAGE, c.slots % PAGE
    c.append(row_pos=c.L.row_pos.clone() if row_pos else None)
    refused()
    others = np.arange(c.rows) != 2
    k[page[others], :, r[others]] = c.dkn[: c.rows][torch.from_numpy(others).cuda()]
    assert torch.equal(c.dk, k)


@pytest.mark.parametrize("bad", [-1, "end", -2 ** 31, 2 ** 31 - 1])
def test_append_reports_slot_positions_outside_the_rope_table(bad):
    c = ChunkCase([20, 7], [4, 9], stale="normal").to_device()
    c.tables()
    at = c.L.row_pos.clone()
    c.L.row_pos[2] = c.max_pos if bad == "end" else bad
    k, page, r = c.dk.clone(), c.slots // PAGE, c.slots % PAGE
    c.append(row_pos=at)
    refused()
    others = np.arange(c.rows) != 2
    k[page[others], :, r[others]] = c.dkn[: c.rows][torch.from_numpy(others).cuda()]
    assert torch.equal(c.dk, k)
