"""GPU tests of the calls that continue a request on the page pool (pcf_chunk_tables, pcf_append_kv,
pcf_chunk_attention) against the fp64 oracle: lengths from nothing to several key tiles, ragged ends,
idle requests, masks, garbage behind every sequence, strides, streams, graphs, refusals on the device,
and the calls together behind a fused prefill."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf
from oracle import chunk, method
from oracle.rope import rotate

from chunk_util import PAGE, ChunkCase, bf16

pytestmark = pytest.mark.gpu

BOUNDS, RANGE = -6, -8


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def check_tables(c):
    assert np.array_equal(c.L.block_table.cpu().numpy(), c.bt)
    assert np.array_equal(c.L.page_pos.cpu().numpy(), c.pp)
    slots, where = c.L.slot_map.cpu().numpy(), c.L.row_pos.cpu().numpy()
    assert np.array_equal(slots[: c.rows], c.slots) and np.all(slots[c.rows:] == -1)
    assert np.array_equal(where[: c.rows], c.where) and np.all(where[c.rows:] == -1)
    assert np.array_equal(c.L.row_base.cpu().numpy(), c.base)
    assert np.array_equal(c.d_seq_out.cpu().numpy(), np.array(c.seq) + np.array(c.new))
    assert c.d_head_out.item() == c.head


# ------------------------------------------------------------------ tables
@pytest.mark.parametrize("seq,new", [
    ([0], [1]), ([0], [16]), ([0], [17]), ([15], [1]), ([15], [2]), ([16], [1]), ([17], [40]), ([5], [0]),
    ([0, 0, 0], [0, 0, 0]), ([1, 16, 31, 0, 64], [3, 0, 1, 33, 16])])
@pytest.mark.parametrize("next_pos", [True, False])
def test_tables(seq, new, next_pos):
    c = ChunkCase(seq, new, spare_rows=3, next_pos=next_pos)
    if not next_pos:      # without tokens a request starts at 0
        c.next_pos = None
    c.to_device()
    c.tables()
    pcf.check_device_error()
    check_tables(c)


@pytest.mark.parametrize("n,hi,spare", [(33, 20, 0), (1000, 3, 50), (1025, 40, 1), (4096, 2, 0), (7, 700, 9)])
def test_tables_of_many_requests(n, hi, spare):
    rng = np.random.default_rng(n)
    c = ChunkCase(rng.integers(0, 60, n).tolist(), rng.integers(0, hi + 1, n).tolist(), hkv=1, hq=1, spare_rows=spare)
    c.to_device()
    c.tables()
    pcf.check_device_error()
    check_tables(c)


def test_tables_leave_unused_entries_alone_and_start_at_the_lists_head():
    c = ChunkCase([20, 0], [13, 1], max_pages=9, extra_pages=9)
    c.table[:, 4:], c.page_pos[:, 4:] = 77, 78
    c.bt, c.pp, c.slots, c.where, c.base, c.head = chunk.tables(c.seq, c.new, c.free, 4, c.table, c.page_pos, c.next_pos)
    c.to_device()
    c.d_head.fill_(4)
    c.tables()
    pcf.check_device_error()
    check_tables(c)


def test_tables_in_place_move_a_captured_loop_on():
    """Lengths and the list's head updated in place: a captured step replayed grows its requests."""
    c = ChunkCase([14, 0, 40], [1, 1, 1], max_pages=8, extra_pages=12)
    c.to_device()
    args = (c.L, c.d_seq, c.d_new, c.d_free, c.d_head, c.d_seq, c.d_head)
    pcf.chunk_tables(*args)                      # (module loading happens outside the capture)
    c.d_seq.copy_(torch.tensor(c.seq)), c.d_head.zero_()
    c.L.block_table.copy_(torch.from_numpy(c.table)), c.L.page_pos.copy_(torch.from_numpy(c.page_pos))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pcf.chunk_tables(*args)
    seq, head, bt, pp = list(c.seq), 0, c.table, c.page_pos
    pos = [int(p) for p in c.next_pos]
    pos[1] = 0                                   # the empty request starts at position 0 without next_pos
    for step in range(40):
        graph.replay()
        bt, pp, slots, where, base, head = chunk.tables(seq, [1, 1, 1], c.free, head, bt, pp, pos)
        assert np.array_equal(c.L.slot_map.cpu().numpy(), slots) and np.array_equal(c.L.row_pos.cpu().numpy(), where)
        seq, pos = [s + 1 for s in seq], [p + 1 for p in pos]
        assert c.d_seq.tolist() == seq and c.d_head.item() == head
    assert np.array_equal(c.L.block_table.cpu().numpy(), bt) and np.array_equal(c.L.page_pos.cpu().numpy(), pp)
    pcf.check_device_error()


REFUSED = {
    "negative length": lambda c: c.d_seq.__setitem__(1, -1),
    "length beyond the table": lambda c: c.d_seq.__setitem__(1, c.max_pages * PAGE + 1),
    "huge length": lambda c: c.d_seq.fill_(2 ** 31 - 1),
    "negative new": lambda c: c.d_new.__setitem__(0, -3),
    "new beyond max_chunk": lambda c: c.d_new.__setitem__(0, c.max_chunk + 1),
    "rows beyond max_rows": lambda c: c.d_new.fill_(c.max_chunk),
    "list runs out": lambda c: c.d_head.fill_(c.d_free.numel()),
    "head behind the list": lambda c: c.d_head.fill_(c.d_free.numel() + 1),
    "negative head": lambda c: c.d_head.fill_(-1),
    "page outside the pool": lambda c: c.d_free.__setitem__(0, c.n_phys),
    "negative page": lambda c: c.d_free.__setitem__(0, -1),
    "position outside the table": lambda c: c.d_next.__setitem__(2, c.max_pos - 3),
    "negative position": lambda c: c.d_next.__setitem__(2, -1),
    "next_pos breaks a started page": lambda c: c.d_next.__setitem__(0, int(c.next_pos[0]) + 1),
    "page position outside the table": lambda c: (c.L.page_pos.__setitem__((0, 1), -100), c.d_next.__setitem__(0, -95)),
}


@pytest.mark.parametrize("what", REFUSED)
def test_refused_lengths_change_nothing_and_stop_the_calls_behind(what):
    c = ChunkCase([21, 3, 0], [2, 5, 17], max_pages=6, max_chunk=20, stale="normal").to_device()
    REFUSED[what](c)
    seq, head = c.d_seq.clone(), c.d_head.clone()
    table, pos, k = c.L.block_table.clone(), c.L.page_pos.clone(), c.dk.clone()
    c.tables()
    c.append()
    c.attend()
    with pytest.raises(pcf.PcfError) as e:
        pcf.check_device_error()
    assert e.value.status == BOUNDS
    assert torch.equal(c.L.block_table, table) and torch.equal(c.L.page_pos, pos)
    assert torch.equal(c.d_seq_out, seq) and torch.equal(c.d_head_out, head)
    assert bool((c.L.slot_map == -1).all()) and bool((c.L.row_pos == -1).all()) and not bool(c.L.row_base.any())
    assert torch.equal(c.dk, k) and bool((c.out == 3.0).all())
    pcf.check_device_error()


def test_total_pages_beyond_the_dims_are_refused():
    c = ChunkCase([40, 40], [1, 1])
    c.to_device()
    c.L = c.layout(max_total_pages=5)             # 3 + 3 pages
    c.tables()
    with pytest.raises(pcf.PcfError):
        pcf.check_device_error()
    c.L = c.layout(max_total_pages=6)
    c.tables()
    pcf.check_device_error()
    check_tables(c)


def test_attention_without_tables_is_refused():
    c = ChunkCase([10], [1]).to_device()
    c.attend()
    with pytest.raises(pcf.PcfError) as e:
        pcf.check_device_error()
    assert e.value.status == BOUNDS and bool((c.out == 3.0).all())


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("shape", [dict(hq=8, hkv=2, d=64), dict(hq=12, hkv=3, d=64), dict(hq=32, hkv=8, d=128)])
@pytest.mark.parametrize("moved", [False, True])
def test_append(shape, moved):
    c = ChunkCase([21, 0, 3, 64], [2, 40, 0, 17], spare_rows=2, **shape).to_device()
    c.tables()
    at = None
    if moved:
        rng = np.random.default_rng(9)
        at = np.concatenate([c.where, [-1, -1]]).astype(np.int32)
        some = rng.random(c.rows) < 0.7
        at[: c.rows][some] = rng.integers(0, c.max_pos, some.sum())
        at[0], at[1] = 0, c.max_pos - 1
    before_k, before_v = c.dk.clone(), c.dv.clone()
    c.append(row_pos=None if at is None else torch.from_numpy(at).cuda())
    pcf.check_device_error()
    page, r = torch.from_numpy(c.slots // PAGE).cuda(), torch.from_numpy(c.slots % PAGE).cuda()
    assert torch.equal(c.dv[page, :, r], c.dvn[: c.rows])
    got = c.dk[page, :, r].float().cpu().double().numpy()
    if moved:
        k = c.k_new[: c.rows].double().numpy()
        exp = chunk.appended(k, c.where, at[: c.rows], c.theta)
        # two products of fp32 angles (2^-24 each), one fp32 sum, one rounding to bf16
        size = np.abs(k) + np.abs(np.roll(k, c.d // 2, axis=-1))
        assert np.all(np.abs(got - exp) <= 2.0 ** -8 * np.abs(exp) + 2.0 ** -21 * size)
        same = at[: c.rows] == c.where
        assert np.array_equal(got[same], k[same])
    else:
        assert torch.equal(c.dk[page, :, r], c.dkn[: c.rows])
    mark = torch.zeros((c.n_phys, PAGE), dtype=torch.bool, device="cuda")
    mark[page, r] = True
    for now, was in ((c.dk, before_k), (c.dv, before_v)):      # every other slot as it was, bit for bit
        keep = ~mark[:, None, :, None].expand_as(now)
        assert torch.equal(now.view(torch.int16)[keep], was.view(torch.int16)[keep])


def test_append_takes_columns_of_a_wider_product():
    c = ChunkCase([5, 30], [20, 4], hq=32, hkv=8, d=128).to_device()
    c.tables()
    wide = torch.zeros((c.max_rows, 48 * 128 + 8), dtype=torch.bfloat16, device="cuda")
    view = wide[:, 8:].view(c.max_rows, 48, 128)
    view[:, 32:40], view[:, 40:] = c.dkn, c.dvn
    pcf.append_kv(c.L, view[:, 32:40], view[:, 40:], c.dk, c.dv)
    pcf.check_device_error()
    page, r = c.slots // PAGE, c.slots % PAGE
    assert torch.equal(c.dk[page, :, r], c.dkn) and torch.equal(c.dv[page, :, r], c.dvn)


def test_append_refuses_positions_outside_the_rope_table():
    c = ChunkCase([5], [4], stale="normal").to_device()
    c.tables()
    for bad in (-1, c.max_pos):
        at = torch.from_numpy(c.where.astype(np.int32)).cuda()
        at[2] = bad
        before = c.dk.clone()
        c.append(row_pos=at)
        with pytest.raises(pcf.PcfError) as e:
            pcf.check_device_error()
        assert e.value.status == BOUNDS
        s = int(c.slots[2])
        assert torch.equal(c.dk[s // PAGE, :, s % PAGE], before[s // PAGE, :, s % PAGE])


# ------------------------------------------------------------------ attention
SHAPES = [dict(hq=8, hkv=2, d=64), dict(hq=32, hkv=8, d=128), dict(hq=12, hkv=3, d=64), dict(hq=24, hkv=12, d=128),
          dict(hq=4, hkv=4, d=64), dict(hq=16, hkv=1, d=128), dict(hq=5, hkv=5, d=128), dict(hq=64, hkv=2, d=64),
          dict(hq=128, hkv=1, d=128), dict(hq=64, hkv=8, d=128)]
IDS = ["{hq}q{hkv}kv{d}".format(**s) for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("seq,new", [
    ([0], [1]), ([1], [1]), ([15], [1]), ([16], [1]), ([127], [1]), ([128], [1]), ([300], [1]),
    ([0, 5, 16, 31, 64, 200], [1, 1, 1, 0, 1, 1]), ([33, 0, 90], [2, 3, 4])])
def test_single_tokens_and_drafts(shape, seq, new):
    c = ChunkCase(seq, new, spare_rows=2, **shape).to_device()
    c.check(c.step())


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("seq,new", [
    ([0], [16]), ([0], [33]), ([7], [64]), ([129], [70]), ([0, 250, 40, 3], [130, 5, 0, 31]),
    ([100, 16], [1, 257])])
def test_chunks(shape, seq, new):
    c = ChunkCase(seq, new, spare_rows=1, **shape).to_device()
    c.check(c.step(), rows=12)


@pytest.mark.parametrize("seq,new,shape", [
    ([4161], [1], dict(hq=32, hkv=8, d=128)), ([9000, 17, 2500], [1, 1, 3], dict(hq=32, hkv=8, d=128)),
    ([3000], [600], dict(hq=32, hkv=8, d=128)), ([2000, 0, 1111, 64], [300, 1, 1, 513], dict(hq=8, hkv=2, d=64)),
    ([5000] * 3, [1] * 3, dict(hq=8, hkv=2, d=64)), ([700], [1024], dict(hq=4, hkv=4, d=64)),
    ([1500, 800], [90, 40], dict(hq=64, hkv=8, d=128))])
def test_longer_contexts(seq, new, shape):
    c = ChunkCase(seq, new, **shape).to_device()
    c.check(c.step(), rows=4)


def test_many_requests():
    rng = np.random.default_rng(12)
    c = ChunkCase(rng.integers(0, 90, 300).tolist(), rng.integers(0, 3, 300).tolist(), hq=8, hkv=2, d=64).to_device()
    c.check(c.step())


def random_excl(c, share, seed):
    rng = np.random.default_rng(seed)
    c.excl = np.zeros((c.n, c.max_pages), dtype=np.uint16)
    for b in range(c.n):
        for j in range(c.seq[b]):
            if rng.random() < share:
                c.excl[b, j // PAGE] |= np.uint16(1 << (j % PAGE))


def poison_excluded(c):
    """Excluded slots hold infinities and NaN (of pages no other request holds)."""
    for b in range(c.n):
        for j in range(c.seq[b]):
            if c.excl[b, j // PAGE] >> (j % PAGE) & 1:
                p = c.table[b, j // PAGE]
                c.k_pool[p, :, j % PAGE] = [float("inf"), float("nan"), -float("inf")][j % 3]
                c.v_pool[p, :, j % PAGE] = [float("nan"), float("inf"), -float("inf")][j % 3]


@pytest.mark.parametrize("n_sms", [1, 2, 5, 23])
@pytest.mark.parametrize("seq_hi,new_hi,shape", [
    (90, 3, dict(hq=8, hkv=2, d=64)), (40, 5, dict(hq=8, hkv=4, d=128)), (400, 4, dict(hq=16, hkv=4, d=128)),
    (90, 60, dict(hq=8, hkv=2, d=64)), (300, 90, dict(hq=32, hkv=4, d=128)), (16, 2, dict(hq=2, hkv=2, d=64))])
def test_few_blocks_with_many_runs_each(n_sms, seq_hi, new_hi, shape):
    """Work dealt to few workers: runs of a page or two, several of them in a worker's share, shares that end
    where a run begins."""
    rng = np.random.default_rng(100 * n_sms + seq_hi)
    n = 40
    c = ChunkCase(rng.integers(0, seq_hi, n).tolist(), rng.integers(0, new_hi, n).tolist(), seed=n_sms, **shape).to_device()
    c.L.dims.n_sms = n_sms
    got = c.step()
    c.check(got)
    first = c.out.clone()
    c.attend()
    pcf.check_device_error()
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("share", [0.0, 0.2])
@pytest.mark.parametrize("kinds", [[3, 20, 16, 60, 1], [20, 3], [16, 16, 33], [5]])
def test_runs_of_one_tile_and_of_more_take_turns(d, share, kinds):
    """Some 480 runs over all blocks, so that a block goes from runs of one row tile to runs of two and back,
    behind lengths that leave the rings at every stage."""
    rng = np.random.default_rng(11)
    n = 120
    c = ChunkCase(rng.integers(0, 700, n).tolist(), [kinds[b % len(kinds)] for b in range(n)], hq=32, hkv=4, d=d, seed=21)
    if share:
        random_excl(c, share, 5)
    got = c.to_device().step()
    for b in range(0, n, 7):
        _, (out, mean_abs, score_abs) = c.oracle(b)
        lim = chunk.attention_bound(out, mean_abs, score_abs)
        bad = ~(np.abs(got[c.base[b]: c.base[b + 1]] - out) <= lim)
        assert not bad.any(), (b, c.seq[b], c.new[b], np.argwhere(bad)[0])
    first = c.out.clone()
    c.attend()
    pcf.check_device_error()
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[5]], ids=[IDS[0], IDS[1], IDS[5]])
@pytest.mark.parametrize("seq,new", [([40, 3, 200], [1, 1, 1]), ([300, 0, 17], [3, 1, 2]), ([150, 290], [70, 140])])
@pytest.mark.parametrize("share", [0.1, 0.5, 1.0])
def test_excluded_slots_take_no_part_whatever_they_hold(shape, seq, new, share):
    c = ChunkCase(seq, new, **shape)
    random_excl(c, share, 5)
    poison_excluded(c)
    c.to_device()
    c.check(c.step(), rows=8)


@pytest.mark.parametrize("seq,new", [([30], [1]), ([30, 140], [3, 1]), ([140, 20], [40, 90])])
def test_rows_with_every_slot_excluded_give_zeros(seq, new):
    c = ChunkCase(seq, new, hq=8, hkv=2, d=64)
    random_excl(c, 1.0, 6)
    n = c.seq[0] + c.new[0]
    for j in range(c.seq[0], n):          # request 0: its new tokens too
        c.excl[0, j // PAGE] |= np.uint16(1 << (j % PAGE))
    poison_excluded(c)
    c.to_device()
    got = c.step()
    assert np.all(got[: c.new[0]] == 0.0)
    c.check(got)


def test_pages_of_another_request_at_other_positions():
    """Three requests over the same physical pages at different positions."""
    c = ChunkCase([96, 96, 96], [1, 20, 2], hq=32, hkv=8, d=128, stale="normal")
    held = 6
    for b in (1, 2):
        c.table[b, :held] = np.roll(c.table[0, :held], b)
    (c.bt, c.pp, c.slots, c.where, c.base, c.head) = chunk.tables(c.seq, c.new, c.free, 0, c.table, c.page_pos,
                                                                  c.next_pos)
    c.to_device()
    c.check(c.step())


def test_spans_with_gaps_between_their_positions():
    c = ChunkCase([128], [3], hq=32, hkv=8, d=128)
    c.max_pos += 3000
    c.page_pos[0, :8] = [700, 716, 3, 19, 35, 2000, 2016, 64]
    c.next_pos = np.array([2500], dtype=np.int32)
    (c.bt, c.pp, c.slots, c.where, c.base, c.head) = chunk.tables(c.seq, c.new, c.free, 0, c.table, c.page_pos,
                                                                  c.next_pos)
    c.to_device()
    c.check(c.step())


@pytest.mark.parametrize("new", [1, 4, 90])
def test_queries_may_be_columns_of_a_wider_product(new):
    c = ChunkCase([100, 60], [new, 1], hq=32, hkv=8, d=128).to_device()
    wide = torch.zeros((c.max_rows, 48, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :32] = c.dq
    c.tables()
    c.append()
    c.attend()
    one = c.out.clone()
    c.dq = wide[:, :32]
    c.out.fill_(3.0)
    c.attend()
    pcf.check_device_error()
    assert torch.equal(one, c.out)
    c.check(c.out.float().cpu().double().numpy(), rows=6)


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [100, 40], [1, 200]])
def test_calls_repeat_bit_for_bit(new):
    c = ChunkCase([700, 333], new, hq=32, hkv=8, d=128).to_device()
    c.step()
    one = c.out.clone()
    for _ in range(3):
        c.out.fill_(3.0)
        c.ws.random_(0, 255)                       # the workspace's contents do not matter
        c.attend()
        pcf.check_device_error()
        assert torch.equal(one, c.out)


def test_pool_offsets_beyond_32_bits():
    """Pages whose elements sit beyond 2^31: 140000 pages x 16384 elements."""
    hq, hkv, d, n_phys = 32, 8, 128, 140000
    c = ChunkCase([40, 20], [1, 70], hq=hq, hkv=hkv, d=d, stale="normal")
    small_k, small_v = c.k_pool, c.v_pool
    ids = np.array([n_phys - 1 - 3 * i for i in range(c.n_phys)], dtype=np.int32)
    dk = torch.empty((n_phys, hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")
    dv = torch.empty_like(dk)
    where = torch.from_numpy(ids).cuda().long()
    dk[where], dv[where] = small_k.cuda(), small_v.cuda()
    old = (c.n_phys, c.table.copy(), c.free.copy())
    c.n_phys, c.table, c.free = n_phys, ids[c.table], ids[c.free]
    c.k_pool, c.v_pool = small_k[:1], small_v[:1]   # (not uploaded: the big pools stand in)
    c.to_device()
    c.dk, c.dv = dk, dv
    got = c.step()
    c.n_phys, c.table, c.free = old
    c.k_pool, c.v_pool = small_k, small_v
    c.check(got, rows=6)


def test_bad_page_and_bad_position_are_reported():
    for new in ([1], [60]):
        for field, value in (("block_table", -1), ("block_table", 10 ** 6), ("page_pos", -1), ("page_pos", 10 ** 6)):
            c = ChunkCase([64], new, hq=32, hkv=8, d=128, stale="normal").to_device()
            c.tables()
            c.append()
            pcf.check_device_error()
            getattr(c.L, field)[0, 1] = value
            c.attend()
            with pytest.raises(pcf.PcfError) as e:
                pcf.check_device_error()
            assert e.value.status == BOUNDS, (new, field, value)


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("which", ["k", "q"])
def test_values_beyond_fp16_are_reported(new, which):
    c = ChunkCase([40], [new], hq=32, hkv=8, d=128, stale="normal")
    if which == "k":
        c.k_pool[c.table[0, 1], 3, 5, 7] = 1e6
    else:
        c.q[0, 9, 11] = 1e8
    c.to_device()
    c.tables()
    c.append()
    c.attend()
    with pytest.raises(pcf.PcfError) as e:
        pcf.check_device_error()
    assert e.value.status == RANGE


@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("which", ["k", "q"])
def test_nan_that_takes_part_is_reported(new, which):
    c = ChunkCase([40], [new], hq=32, hkv=8, d=128, stale="normal")
    if which == "k":
        c.k_pool[c.table[0, 1], 3, 5, 7] = float("nan")
    else:
        c.q[0, 9, 99] = float("nan")
    c.to_device()
    c.tables()
    c.append()
    c.attend()
    with pytest.raises(pcf.PcfError) as e:
        pcf.check_device_error()
    assert e.value.status == RANGE


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 1e6, -1e6, 65280.0])
@pytest.mark.parametrize("chunk_at", [0, 7, 8, 15])
def test_keys_of_runs_of_one_tile_are_checked(value, chunk_at):
    """65280 is the largest bf16 that fp16 holds; the key sits at position 0, where it is not turned."""
    c = ChunkCase([40], [20], hq=32, hkv=8, d=128, stale="normal", pos0=0)
    c.k_pool[c.table[0, 0], 3, 0] = 0.0
    c.k_pool[c.table[0, 0], 3, 0, 8 * chunk_at + 3] = value
    c.to_device()
    c.tables()
    c.append()
    c.attend()
    if value == 65280.0:
        pcf.check_device_error()
        return
    with pytest.raises(pcf.PcfError) as e:
        pcf.check_device_error()
    assert e.value.status == RANGE


@pytest.mark.parametrize("seq,new", [([40], [1]), ([40], [3]), ([40], [60]), ([40], [200]), ([3000], [1]),
                                     ([3000], [200]), ([9, 70, 500], [2, 40, 1])])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_and_take_part_are_reported(seq, new, value):
    """In a cached page, and in the last new token's value, which earlier rows do not see."""
    for where in ("page", "new"):
        c = ChunkCase(seq, new, hq=32, hkv=8, d=128, stale="normal")
        if where == "page":
            c.v_pool[c.table[-1, 0], 5, 6, 77] = value
        else:
            c.v_new[c.rows - 1, 2, 9] = value
        c.to_device()
        c.tables()
        c.append()
        c.attend()
        with pytest.raises(pcf.PcfError) as e:
            pcf.check_device_error()
        assert e.value.status == RANGE, where


def test_plan_of_other_dims_is_refused():
    for new in ([1], [60]):
        c = ChunkCase([40], new, hq=32, hkv=8, d=128, stale="normal", spare_rows=70).to_device()
        c.tables()
        c.append()
        plan = c.L.plan.clone()
        other = pcf.ChunkLayout(1, 32, 8, 128, c.n_phys, c.max_pos, max_pages=c.max_pages, max_rows=c.max_rows,
                                max_chunk=new[0] + 1)
        other.block_table, other.page_pos = c.L.block_table, c.L.page_pos
        other.row_pos = c.L.row_pos
        other.plan[: plan.numel()] = plan[: other.plan.numel()]
        ws = torch.empty(other.attention_workspace_bytes() + 16, dtype=torch.uint8, device="cuda")
        pcf.chunk_attention(other, c.dq, c.dk, c.dv, c.rope, c.out, ws)
        with pytest.raises(pcf.PcfError) as e:
            pcf.check_device_error()
        assert e.value.status == BOUNDS and bool((c.out == 3.0).all())


def test_idle_batch_writes_nothing():
    c = ChunkCase([40, 0], [0, 0], spare_rows=4).to_device()
    c.step()
    assert bool((c.out == 3.0).all())


def test_side_stream():
    c = ChunkCase([200, 40], [1, 60], hq=32, hkv=8, d=128).to_device()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.tables(stream=s)
    c.append(stream=s)
    c.attend(stream=s)
    pcf.check_device_error(s)
    torch.cuda.current_stream().wait_stream(s)
    c.check(c.out.float().cpu().double().numpy(), rows=8)


def test_two_streams_at_once_with_a_workspace_each():
    cs = [ChunkCase([1500, 40 + i], [1, 30 + 50 * i], hq=32, hkv=8, d=128, seed=i).to_device() for i in range(2)]
    for c in cs:
        c.tables()
        c.append()
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            c.attend(stream=s)
    torch.cuda.synchronize()
    pcf.check_device_error()
    for c in cs:
        c.check(c.out.float().cpu().double().numpy(), rows=5)


def merged_oracle(q, q_pos, K, V, k_pos, theta):
    """Attention over keys given with their true positions (order and tables play no part)."""
    n = len(k_pos)
    return chunk.attention(q, q_pos, K, V, k_pos, np.ones((q.shape[0], n), dtype=bool), theta)


@pytest.mark.parametrize("shape", [dict(hq=8, hkv=2, d=64, theta=1e4), dict(hq=32, hkv=8, d=128, theta=5e5)])
def test_a_fused_batch_decodes_on(shape):
    """Score, select and fuse a batch over shared spans; move its recomputed and query tokens into
    pages of their own; decode several tokens and then a chunk, as a captured step where one token is
    taken; every output against attention over the merged cache at the true positions."""
    from workload import small_custom_batch
    from gpu_util import GpuBatch, assert_close_out
    spans = [[(0, 3, 7, 5), (6, 2, 55, 9)], [(6, 2, 100, 3), (0, 3, 132, 0)], [(3, 1, 0, 16)]]
    b = small_custom_batch(spans[0], 6, n_phys_pages=60, extra_requests=[(spans[1], 21, 180), (spans[2], 1, 16)],
                           **shape)
    gb = GpuBatch(b)
    gb.score()
    gb.topk()
    gb.attention()
    hq, hkv, d, theta = b.hq, b.hkv, b.d, shape["theta"]
    n = len(b.requests)
    rows = [r.n_rows for r in b.requests]
    sel = gb.cf.sel_idx[: gb.L.total_sel].cpu().numpy()
    # every request's merged cache at its true positions, on the host
    merged = []
    for i, r in enumerate(b.requests):
        _, K, V, kpos = gb.oracle_request(i)
        mine = sel[gb.sel_base[i]: gb.sel_base[i] + r.n_rows - r.n_query]
        keep = np.setdiff1d(np.arange(len(kpos)), mine)
        sl = slice(gb.row_base[i], gb.row_base[i] + r.n_rows)
        pos = method.row_positions(mine, kpos, r.n_query, r.query_pos0)
        merged.append([np.concatenate([K[keep], b.k_fresh[sl].double().numpy()]),
                       np.concatenate([V[keep], b.v_fresh[sl].double().numpy()]),
                       np.concatenate([kpos[keep], pos])])
    max_pos, max_pages = 400, 16
    rope = pcf.rope_table(d, theta, max_pos).cuda()
    free = torch.arange(59, 10, -1, dtype=torch.int32, device="cuda")
    head = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    seq = i32([r.n_cached for r in b.requests])
    k_pool, v_pool = gb.k_pool.clone(), gb.v_pool.clone()
    # the fused rows into pages of their own: the recomputed tokens take the slots before the query's
    L0, excl = pcf.ChunkLayout.from_layout(gb.L, max_pages=max_pages, max_rows=sum(rows), max_chunk=max(rows),
                                           max_pos=max_pos, excl=gb.cf.excl)
    start = i32([r.query_pos0 - (r.n_rows - r.n_query) for r in b.requests])
    pcf.chunk_tables(L0, seq, i32(rows), free, head, seq, head, next_pos=start)
    pcf.append_kv(L0, gb.k_fresh, gb.v_fresh, k_pool, v_pool, rope=rope, row_pos=gb.cf.row_pos)
    pcf.check_device_error()
    pages = slice(0, 10)
    assert torch.equal(k_pool[pages], gb.k_pool[pages])          # the shared pages stay as they were

    def layout(max_rows, max_chunk):
        L = pcf.ChunkLayout(n, hq, hkv, d, 60, max_pos, max_pages=max_pages, max_rows=max_rows, max_chunk=max_chunk)
        L.block_table, L.page_pos = L0.block_table, L0.page_pos
        return L

    g = torch.Generator().manual_seed(11)
    pos = [r.query_pos0 + r.n_query for r in b.requests]

    def check(new, out, q, k, v):
        base = 0
        for i in range(n):
            for t in range(new[i]):
                # the key as the pool holds it: moved keys carry one more rounding, within the bound
                # below; new ones none
                m = merged[i]
                m[0] = np.concatenate([m[0], k[base: base + 1].double().numpy()])
                m[1] = np.concatenate([m[1], v[base: base + 1].double().numpy()])
                m[2] = np.concatenate([m[2], [pos[i]]])
                o, mean_abs, score_abs = merged_oracle(q[base: base + 1].double().numpy(), [pos[i]], *m, theta)
                lim = chunk.attention_bound(o, mean_abs, score_abs)
                # stored keys rounded once more, half a bf16 step: scores off by 2^-8 sum |q k| at most
                lim = lim + 2.1 * 2.0 ** -8 * score_abs[..., None] * mean_abs
                assert np.all(np.abs(out[base] - o[0]) <= lim[0]), (i, t)
                pos[i], base = pos[i] + 1, base + 1

    # decode: one captured step, replayed
    L = layout(n, 1)
    new = i32([1] * n)
    q, k, v = (torch.zeros((n, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    out = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, L.attention_workspace_bytes()), dtype=torch.uint8, device="cuda")

    def step():
        pcf.chunk_tables(L, seq, new, free, head, seq, head)
        pcf.append_kv(L, k, v, k_pool, v_pool)
        pcf.chunk_attention(L, q, k_pool, v_pool, rope, out, ws, excl=excl)

    def draws():
        hs = [bf16(g, n, h, d) for h in (hq, hkv, hkv)]
        for dst, src in zip((q, k, v), hs):
            dst.copy_(src)
        return hs

    hs = draws()
    step()                                         # (also loads the kernels)
    pcf.check_device_error()
    check([1] * n, out.float().cpu().double().numpy(), *hs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(18):
        hs = draws()
        graph.replay()
        pcf.check_device_error()
        check([1] * n, out.float().cpu().double().numpy(), *hs)
    # then a chunk for two of them
    new = [40, 0, 3]
    L = layout(43, 40)
    q, k, v = bf16(g, 43, hq, d), bf16(g, 43, hkv, d), bf16(g, 43, hkv, d)
    out = torch.zeros((43, hq, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, L.attention_workspace_bytes()), dtype=torch.uint8, device="cuda")
    pcf.chunk_tables(L, seq, i32(new), free, head, seq, head)
    pcf.append_kv(L, k.cuda(), v.cuda(), k_pool, v_pool)
    pcf.chunk_attention(L, q.cuda(), k_pool, v_pool, rope, out, ws, excl=excl)
    pcf.check_device_error()
    check(new, out.float().cpu().double().numpy(), q, k, v)


def test_two_captured_graphs_share_a_workspace_in_order():
    """Two graphs that use one workspace, replayed one behind the other."""
    a = ChunkCase([900, 20], [1, 1], hq=32, hkv=8, d=128, seed=1).to_device()
    b = ChunkCase([30, 500], [70, 1], hq=32, hkv=8, d=128, seed=2).to_device()
    ws = torch.empty(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    a.ws = b.ws = ws
    graphs = []
    for c in (a, b):
        c.step()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.tables()
            c.append()
            c.attend()
        graphs.append(gr)
    a.out.fill_(3.0), b.out.fill_(3.0)
    for _ in range(4):
        for gr in graphs:
            gr.replay()
    pcf.check_device_error()
    for c in (a, b):
        c.check(c.out.float().cpu().double().numpy(), rows=6)


@pytest.mark.parametrize("seq,new", [([300], [1]), ([40, 3], [1, 1]), ([2000], [2]), ([30, 900], [70, 1])])
def test_a_workspace_full_of_nan_does_not_matter(seq, new):
    """Partial results that a call has not written must not be read, not even with weight zero."""
    c = ChunkCase(seq, new, hq=32, hkv=8, d=128).to_device()
    c.tables()
    c.append()
    c.ws.fill_(255)
    c.attend()
    pcf.check_device_error()
    c.check(c.out.float().cpu().double().numpy(), rows=6)


@pytest.mark.parametrize("extra", [[], ["--tokens", "3"], ["--tokens", "40"]])
def test_bench_decode_runs_behind_the_fused_prefill(extra):
    import json
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "bench.py", "--config", "tiny", "--op", "decode", "--steps", "3", "--warmup", "3"]
                       + extra, cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["op"] == "decode" and line["value"] > 0 and line["roofline"]["algorithmic_bytes_per_launch"] > 0


@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[0], SHAPES[8]], ids=[IDS[1], IDS[0], IDS[8]])
def test_requests_of_every_kind_in_one_batch(shape):
    """Idle requests, single tokens, drafts, chunks of one row tile and of several, with exclusions."""
    c = ChunkCase([700, 31, 0, 260, 900, 1, 145, 16], [1, 0, 33, 3, 150, 5, 20, 2], spare_rows=3, **shape)
    random_excl(c, 0.2, 3)
    poison_excluded(c)
    c.to_device()
    c.check(c.step(), rows=6)
