"""GPU tests of the calls that check a tree of drafted tokens (pcf_tree_tables, pcf_tree_attention,
pcf_tree_accept, pcf_tree_keep) against the fp64 oracle: trees from one node to 256, chains, stars and random
ones, contexts from nothing to long ones, masks, garbage behind every sequence, strides, streams, graphs,
refusals on the device, and the calls together over many steps."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf
from oracle import chunk, tree

from chunk_long import NORM, outside, planted_key, planted_value
from chunk_util import PAGE, bf16
from tree_util import TreeCase, chain, random_tree, star

pytestmark = pytest.mark.gpu

BOUNDS, RANGE = -6, -8
SHAPES = [dict(hq=8, hkv=2, d=64), dict(hq=32, hkv=8, d=128), dict(hq=64, hkv=8, d=128), dict(hq=4, hkv=4, d=64),
          dict(hq=16, hkv=1, d=128), dict(hq=24, hkv=12, d=128), dict(hq=128, hkv=1, d=64)]
IDS = ["-".join(str(v) for v in s.values()) for s in SHAPES]


@pytest.fixture(autouse=True)
def clean_error_word():
    pcf.check_device_error()
    yield


def raises(status):
    with pytest.raises(pcf.PcfError) as e:
        pcf.check_device_error()
    assert e.value.status == status


def trees(sizes, seed=0, width=None, roots=False):
    rng = np.random.default_rng(seed)
    return [random_tree(n, rng, width, roots) for n in sizes]


def check_tables(c):
    pos, seen = c.tree.row_pos.cpu().numpy(), c.tree.seen.cpu().numpy().view(np.uint32)
    assert np.array_equal(pos[: c.rows], c.node_pos) and np.all(pos[c.rows:] == -1)
    assert np.array_equal(seen[: c.rows], c.bits) and not seen[c.rows:].any()


def check_accepted(c):
    path, kept, token, length, free, head = c.accepted()
    assert c.tree.path.tolist() == path + [-1] * (c.max_rows - c.rows)
    assert c.tree.n_kept.tolist() == kept and c.tree.next_token.tolist() == token
    assert c.d_seq_out.tolist() == length and c.d_head_out.item() == head and c.d_free.tolist() == [int(x) for x in free]


# ------------------------------------------------------------------ tables
@pytest.mark.parametrize("sizes", [[1], [2], [31], [32], [33], [64], [65], [255], [256], [0], [0, 0], [7, 0, 256, 1, 40]])
@pytest.mark.parametrize("kind", ["chain", "star", "random", "narrow", "roots"])
def test_tables(sizes, kind):
    parents = {"chain": [chain(n) for n in sizes], "star": [star(n) if n else [] for n in sizes],
               "random": trees(sizes, 1), "narrow": trees(sizes, 2, 4), "roots": trees(sizes, 3, None, True)}[kind]
    c = TreeCase([3 + 5 * b for b in range(len(sizes))], parents, spare_rows=5).to_device()
    c.tables()
    pcf.check_device_error()
    check_tables(c)
    c.tables()                                     # the same call again
    pcf.check_device_error()
    check_tables(c)


def test_tables_of_many_requests():
    rng = np.random.default_rng(5)
    c = TreeCase(rng.integers(0, 60, 4096), trees(rng.integers(0, 12, 4096), 4), max_chunk=70).to_device()
    c.tables()
    pcf.check_device_error()
    check_tables(c)


@pytest.mark.parametrize("row,value", [(0, 0), (0, -2), (3, 3), (5, 99), (40, 40), (40, -2 ** 31), (44, 2 ** 31 - 1)])
def test_parents_out_of_range_are_reported(row, value):
    c = TreeCase([20, 7], trees([41, 5])).to_device()
    c.d_parent[row] = value
    c.tables()
    raises(BOUNDS)
    c.append()
    c.attend()                                     # (defined for any parents: such a node begins at the held tokens)
    pcf.check_device_error()
    c.accept()
    raises(BOUNDS)


def test_refused_lengths_leave_no_rows():
    c = TreeCase([20, 7], trees([20, 5])).to_device()
    c.d_next[0] += 1                               # breaks a started page
    c.tables()
    raises(BOUNDS)
    assert bool((c.tree.row_pos == -1).all()) and not bool(c.tree.seen.any())
    free = c.d_free.clone()
    c.append()
    c.attend()
    c.accept()
    pcf.tree_keep(c.L, c.tree, [c.dk], [c.dv])
    pcf.check_device_error()
    assert bool((c.out == 3.0).all()) and c.tree.n_kept.tolist() == [0, 0] and bool((c.tree.path == -1).all())
    assert c.d_seq_out.tolist() == [20, 7] and c.d_head_out.item() == 0 and torch.equal(c.d_free, free)


def test_plans_of_other_dims_are_refused():
    c = TreeCase([40], trees([20]), stale="normal").to_device()
    c.tables()
    c.append()
    pcf.check_device_error()
    d = TreeCase([40], trees([20]), stale="normal", max_chunk=20, extra_pages=4).to_device()
    d.L.plan[: c.L.plan.numel()] = c.L.plan
    pcf.tree_tables(d.L, d.tree, d.d_parent)
    raises(BOUNDS)
    assert bool((d.tree.row_pos == -1).all())
    d.attend()                                     # (a plan without rows)
    pcf.check_device_error()
    assert bool((d.out == 3.0).all())
    d.tables()
    pcf.check_device_error()
    d.tree.plan[: c.tree.plan.numel()] = c.tree.plan
    for call in (d.attend, d.accept, lambda: pcf.tree_keep(d.L, d.tree, [d.dk], [d.dv])):
        k = d.dk.clone()
        call()
        raises(BOUNDS)
        assert torch.equal(d.dk, k) or bool(torch.isnan(k).any())
    assert bool((d.out == 3.0).all())


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("seq,sizes", [
    ([0], [1]), ([5], [1]), ([0], [7]), ([16], [16]), ([63], [1]), ([64], [2]), ([61], [9]), ([127], [26]), ([129], [31]),
    ([300], [64]), ([40, 0, 500, 17], [5, 3, 33, 0])])
def test_attention(shape, seq, sizes):
    c = TreeCase(seq, trees(sizes, sum(seq)), spare_rows=2, seed=sum(seq) + 3, **shape).to_device()
    c.check(c.step(), rows=8)


@pytest.mark.parametrize("kind", ["chain", "star", "random", "roots"])
@pytest.mark.parametrize("sizes", [[256], [200, 7, 130], [65, 64, 63], [33]])
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[2]], ids=[IDS[0], IDS[2]])
def test_large_trees(shape, sizes, kind):
    parents = {"chain": [chain(n) for n in sizes], "star": [star(n) for n in sizes], "random": trees(sizes, 6, 50),
               "roots": trees(sizes, 7, None, True)}[kind]
    c = TreeCase([90, 13, 200][: len(sizes)], parents, seed=9, **shape).to_device()
    c.check(c.step(), rows=8)


def test_a_chain_is_a_chunk():
    """The same tokens as a line: both calls within the oracle's bounds, so near one another."""
    c = TreeCase([700, 90, 3], [chain(40), chain(1), chain(130)], hq=32, hkv=8, d=128).to_device()
    got = c.step()
    c.check(got, rows=8)
    ws = torch.empty(max(16, c.L.attention_workspace_bytes()), dtype=torch.uint8, device="cuda")
    line = torch.full_like(c.out, 3.0)
    pcf.chunk_attention(c.L, c.dq, c.dk, c.dv, c.rope, line, ws)
    pcf.check_device_error()
    c.check(line.float().cpu().double().numpy(), rows=8)


def random_excl(c, share, seed):
    rng = np.random.default_rng(seed)
    c.excl = np.zeros((c.n, c.max_pages), dtype=np.uint16)
    for b in range(c.n):
        for j in range(c.seq[b]):
            if rng.random() < share:
                c.excl[b, j // PAGE] |= np.uint16(1 << (j % PAGE))


def poison_excluded(c, value=float("nan")):
    for b in range(c.n):
        for j in range(c.seq[b] + c.new[b]):
            if c.excl[b, j // PAGE] >> (j % PAGE) & 1:
                for pool, rows in ((c.k_pool, c.k_new), (c.v_pool, c.v_new)):
                    if j >= c.seq[b]:
                        rows[c.base[b] + j - c.seq[b]] = value
                    else:
                        pool[c.bt[b, j // PAGE], :, j % PAGE] = value


@pytest.mark.parametrize("shape", SHAPES[:4], ids=IDS[:4])
@pytest.mark.parametrize("share", [0.1, 0.9, 1.0])
@pytest.mark.parametrize("sizes", [[3, 40, 1, 0], [17, 90, 2, 140]])
def test_excluded_slots_may_hold_anything(shape, share, sizes):
    c = TreeCase([300, 31, 64, 150], trees(sizes, 8), seed=4, **shape)
    random_excl(c, share, 5)
    poison_excluded(c, float("nan") if share < 1 else float("inf"))
    c.to_device()
    c.check(c.step(), rows=8)


def test_rows_with_nothing_left_give_zeros():
    """Every held slot and some nodes excluded: a node whose whole line is gives zeros."""
    for sizes, shape in (([6, 70], SHAPES[0]), ([6, 70], SHAPES[2])):
        c = TreeCase([40, 100], trees(sizes, 2), **shape)
        random_excl(c, 1.0, 1)
        for b in range(2):
            for u in (0, 1, 3):
                j = c.seq[b] + u
                c.excl[b, j // PAGE] |= np.uint16(1 << (j % PAGE))
        poison_excluded(c)
        c.to_device()
        got = c.step()
        c.check(got)
        for b in range(2):
            gone = [t for t, line in enumerate(tree.lines(c.parents[b])) if set(line) <= {0, 1, 3}]
            assert gone and not got[c.base[b] + np.array(gone)].any()


def test_lowest_values_and_large_scores():
    """Keys whose scores are far below the others' all over a request, and far above them in one place."""
    c = TreeCase([200, 90], trees([20, 5], 3), hq=32, hkv=8, d=128, stale="normal")
    c.k_pool[c.table[0, 3], :, 5] *= 40
    c.k_pool[c.table[1]] *= 0.01
    c.to_device()
    c.check(c.step(), rows=6)


def test_strided_queries_and_rows_behind_the_last():
    c = TreeCase([120, 33], trees([9, 40], 3), hq=32, hkv=8, d=128, spare_rows=3).to_device()
    wide = torch.zeros((c.max_rows, 48, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :32], wide[:, 32:40], wide[:, 40:] = c.dq, c.dkn, c.dvn
    c.dq, c.dkn, c.dvn = wide[:, :32], wide[:, 32:40], wide[:, 40:]
    c.check(c.step(), rows=8)


@pytest.mark.parametrize("n_sms", [1, 2, 3, 37])
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1]], ids=IDS[:2])
def test_any_number_of_blocks(n_sms, shape):
    c = TreeCase([300, 0, 40, 900, 77, 64], trees([3, 40, 1, 33, 130, 16], 9, 9), seed=n_sms, **shape)
    random_excl(c, 0.2, 2)
    poison_excluded(c)
    c.to_device()
    c.L.dims.n_sms = n_sms
    got = c.step()
    first = c.out.clone()
    for _ in range(10):
        c.out.fill_(3.0)
        c.ws.fill_(255)                            # the workspace's contents do not matter
        c.attend()
        pcf.check_device_error()
        assert torch.equal(c.out, first)
    c.check(got, rows=8)


@pytest.mark.parametrize("seq,sizes,shape", [
    ([9000], [26], dict(hq=32, hkv=8, d=128)), ([33000], [64], dict(hq=8, hkv=2, d=64)),
    ([9000, 17, 2500], [4, 100, 30], dict(hq=32, hkv=8, d=128)), ([16000], [1], dict(hq=32, hkv=8, d=128))])
@pytest.mark.parametrize("n_sms", [None, 3])
def test_no_page_is_lost_or_counted_twice(seq, sizes, shape, n_sms):
    """Keys with about half of a row's weight, planted at the borders of the context, of the blocks' shares and
    of key tiles; and the norm of every row's error."""
    c = TreeCase(seq, trees(sizes, 5, 6), seed=sum(seq), stale="normal", **shape).to_device()
    if n_sms is not None:
        c.L.dims.n_sms = n_sms
    c.tables()
    pcf.check_device_error()
    blocks = c.L.dims.n_sms
    plan = c.tree.plan.cpu().numpy()
    at = (4 + 4 * (c.n + 1) + 3) // 4 * 4
    shares = plan[at: at + 12 * blocks].reshape(blocks, 12)
    rng = np.random.default_rng(3)
    g = c.hq // c.hkv
    picked = []
    for b in range(c.n):
        borders = sorted({x for s in shares if s[0] == b and s[4] > 0 for x in (4 * int(s[3]) - 1, 4 * int(s[3])) if x >= 0})
        rng.shuffle(borders)
        pages = [0, max(0, c.seq[b] // PAGE - 1), 3, 4, 7, 8] + borders[:40] + rng.integers(0, c.seq[b] // PAGE + 1, 8).tolist()
        rows = sorted({0, c.new[b] - 1, *rng.integers(0, c.new[b], 3)})
        used = [set() for _ in range(c.hkv)]
        i = 0
        for t in rows:
            for h in range(c.hq):
                p = pages[i % len(pages)]
                free = [j for j in range(p * PAGE, min((p + 1) * PAGE, c.seq[b])) if j not in used[h // g]]
                i += 1
                if not free:
                    continue
                j = free[(7 * i) % len(free)]
                used[h // g].add(j)
                pos = int(c.pp[b, j // PAGE]) + j % PAGE
                key = planted_key(c.q[c.base[b] + t, h].double().numpy(), int(c.node_pos[c.base[b] + t]), pos, c.seq[b],
                                  c.theta)
                c.k_pool[c.bt[b, j // PAGE], h // g, j % PAGE] = torch.from_numpy(key).to(torch.bfloat16)
                c.v_pool[c.bt[b, j // PAGE], h // g, j % PAGE] = torch.from_numpy(planted_value(c.d, i)).to(torch.bfloat16)
        picked.append(rows)
    c.dk.copy_(c.k_pool), c.dv.copy_(c.v_pool)
    c.append()
    c.attend()
    pcf.check_device_error()
    got = c.out.float().cpu().double().numpy()
    for b in range(c.n):
        t, exact = c.oracle(b, picked[b])
        wrong = outside(got[c.base[b] + t], *exact)
        assert wrong is None, (b, c.seq[b], c.new[b], wrong)


@pytest.mark.parametrize("sizes", [[1], [3], [20], [70]])
def test_bad_page_and_bad_position_are_reported(sizes):
    for field, value in (("block_table", -1), ("block_table", 10 ** 6), ("page_pos", -1), ("page_pos", 10 ** 6),
                         ("row_pos", -1), ("row_pos", 10 ** 6)):
        c = TreeCase([64], trees(sizes), hq=32, hkv=8, d=128, stale="normal").to_device()
        c.tables()
        c.append()
        pcf.check_device_error()
        if field == "row_pos":
            c.tree.row_pos[sizes[0] - 1] = value
        else:
            getattr(c.L, field)[0, 1] = value
        c.attend()
        raises(BOUNDS)


@pytest.mark.parametrize("sizes", [[1], [3], [20], [70]])
@pytest.mark.parametrize("which", ["k", "q", "k_new", "v", "v_new"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 1e8])
def test_what_is_not_finite_and_takes_part_is_reported(sizes, which, value):
    c = TreeCase([40], trees(sizes), hq=32, hkv=8, d=128, stale="normal")
    n = sizes[0]
    if which == "k":
        c.k_pool[c.table[0, 1], 3, 5, 7] = value
    elif which == "v":
        c.v_pool[c.table[0, 0], 5, 6, 77] = value
    elif which == "q":
        c.q[n - 1, 9, 99] = value
    elif which == "k_new":
        c.k_new[n - 1, 7, 127] = value
    else:
        c.v_new[n - 1, 2, 9] = value
    c.to_device()
    c.tables()
    c.append()
    c.attend()
    if value == 1e8 and which.startswith("v"):     # (a value may be as large as bf16 holds)
        pcf.check_device_error()
    else:
        raises(RANGE)


@pytest.mark.parametrize("value", [65280.0, -65280.0, 65536.0])
@pytest.mark.parametrize("at", [0, 8, 63, 64, 127])
def test_the_largest_keys_fp16_holds(value, at):
    """65280 is the largest bf16 that fp16 holds; the key sits at position 0, where it is not turned."""
    c = TreeCase([40], trees([20]), hq=32, hkv=8, d=128, stale="normal", pos0=0)
    c.k_pool[c.table[0, 0], 3, 0] = 0.0
    c.k_pool[c.table[0, 0], 3, 0, at] = value
    c.to_device()
    c.tables()
    c.append()
    c.attend()
    if abs(value) == 65280.0:
        pcf.check_device_error()
    else:
        raises(RANGE)


def test_pool_offsets_beyond_32_bits():
    """Pages whose elements sit beyond 2^31: 140000 pages x 16384 elements."""
    hq, hkv, d, n_phys = 32, 8, 128, 140000
    c = TreeCase([40, 20], trees([26, 70], 3), hq=hq, hkv=hkv, d=d, stale="normal")
    small_k, small_v = c.k_pool, c.v_pool
    ids = np.array([n_phys - 1 - 3 * i for i in range(c.n_phys)], dtype=np.int32)
    dk = torch.empty((n_phys, hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")
    dv = torch.empty_like(dk)
    where = torch.from_numpy(ids).cuda().long()
    dk[where], dv[where] = small_k.cuda(), small_v.cuda()
    old = (c.n_phys, c.table.copy(), c.free.copy(), c.bt.copy(), c.slots.copy())
    c.n_phys, c.table, c.free = n_phys, ids[c.table], ids[c.free]
    c.k_pool, c.v_pool = small_k[:1], small_v[:1]  # (not uploaded: the big pools stand in)
    c.to_device()
    c.dk, c.dv = dk, dv
    got = c.step()
    c.n_phys, c.table, c.free, c.bt, c.slots = old
    c.k_pool, c.v_pool = small_k, small_v
    c.check(got, rows=6)
    # and the branches kept there
    c.accept()
    before = [t[where].clone() for t in (dk, dv)]
    pcf.tree_keep(c.L, c.tree, [dk], [dv])
    pcf.check_device_error()
    path, kept = c.accepted()[:2]
    for t, b in zip((dk, dv), before):
        want = tree.keep(b.float().cpu().numpy(), c.seq, c.base, path, kept, c.bt)
        assert np.array_equal(t[where].float().cpu().numpy(), want)


def test_side_stream_and_two_at_once():
    cs = [TreeCase([1500, 40 + i], trees([26, 30 + 50 * i], i), hq=32, hkv=8, d=128, seed=i).to_device() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            c.tables(stream=s)
            c.append(stream=s)
            c.attend(stream=s)
            c.accept(stream=s)
    torch.cuda.synchronize()
    pcf.check_device_error()
    for c in cs:
        c.check(c.out.float().cpu().double().numpy(), rows=5)
        check_accepted(c)


# ------------------------------------------------------------------ accept, keep
@pytest.mark.parametrize("sizes", [[1], [2], [40], [256], [0], [5, 0, 33, 64, 7], [256, 200, 1]])
@pytest.mark.parametrize("roots", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 50])
def test_accept(sizes, roots, vocab):
    c = TreeCase([14 + 3 * b for b in range(len(sizes))], trees(sizes, vocab, 6, roots), vocab=vocab, roots=roots,
                 spare_rows=4).to_device()
    c.tables()
    for _ in range(2):                             # (the second call finds what the first one left)
        c.accept()
        pcf.check_device_error()
        check_accepted(c)


def test_accept_of_a_long_chain_and_of_many_requests():
    c = TreeCase([5], [chain(256)], vocab=1).to_device()
    c.tables()
    c.accept()
    pcf.check_device_error()
    assert c.tree.n_kept.tolist() == [256]
    check_accepted(c)
    rng = np.random.default_rng(5)
    c = TreeCase(rng.integers(0, 60, 4096), trees(rng.integers(0, 20, 4096), 4, 3), vocab=2).to_device()
    c.tables()
    for _ in range(3):
        c.accept()
        pcf.check_device_error()
        check_accepted(c)


def test_accept_takes_the_list_back_in_place():
    """Lengths and head that the tables moved on in place are set to the branches'; the next step starts there."""
    c = TreeCase([14, 30], trees([40, 20], 3, 4), vocab=2).to_device()
    c.d_seq_out, c.d_head_out = c.d_seq, c.d_head
    c.tables()
    assert c.d_seq.tolist() == [54, 50]
    c.accept()
    pcf.check_device_error()
    check_accepted(c)


def test_accept_refuses_a_list_shorter_than_what_was_taken():
    c = TreeCase([14], trees([40], 3)).to_device()
    c.tables()
    pcf.check_device_error()
    c.d_free = c.d_free[: c.head - 1].clone()
    before = c.d_free.clone()
    c.accept()
    raises(BOUNDS)
    assert torch.equal(c.d_free, before)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("layers", [1, 3])
def test_keep(shape, layers):
    c = TreeCase([0, 14, 31, 40, 7], trees([20, 33, 1, 0, 70], 3, 4), vocab=2, **shape).to_device()
    c.tables()
    c.append()
    c.accept()
    pcf.check_device_error()
    path, kept = c.accepted()[:2]
    g = torch.Generator().manual_seed(4)
    pools = [bf16(g, *c.dk.shape).cuda() for _ in range(2 * layers)]
    before = [p.float().cpu().numpy() for p in pools]
    pcf.tree_keep(c.L, c.tree, pools[:layers], pools[layers:])
    pcf.check_device_error()
    for p, b in zip(pools, before):
        assert np.array_equal(p.float().cpu().numpy(), tree.keep(b, c.seq, c.base, path, kept, c.bt))


def test_keep_of_more_layers_than_a_launch_takes():
    c = TreeCase([14, 3], trees([33, 12], 3, 4), vocab=2, stale="normal").to_device()
    c.tables()
    c.accept()
    path, kept = c.accepted()[:2]
    pools = torch.randn((2 * 131,) + tuple(c.dk.shape), device="cuda").to(torch.bfloat16)
    before = pools.float().cpu().numpy()
    pcf.tree_keep(c.L, c.tree, list(pools[:131]), list(pools[131:]))
    pcf.check_device_error()
    for l in (0, 63, 64, 127, 128, 130, 131, 200, 261):
        assert np.array_equal(pools[l].float().cpu().numpy(), tree.keep(before[l], c.seq, c.base, path, kept, c.bt))


@pytest.mark.parametrize("path,kept", [([5, 0, 2], 3), ([0, 33], 2), ([0, -1], 2), ([0, 2 ** 31 - 1], 2), ([0, 1], 34),
                                       ([0, 1], -1)])
def test_keep_refuses_paths_that_are_none(path, kept):
    c = TreeCase([14], trees([33], 3), stale="normal").to_device()
    c.tables()
    c.append()
    pcf.check_device_error()
    c.tree.path[: len(path)] = torch.tensor(path, dtype=torch.int32, device="cuda")
    c.tree.n_kept.fill_(kept)
    pcf.tree_keep(c.L, c.tree, [c.dk], [c.dv])
    raises(BOUNDS)


def test_keep_reports_pages_outside_the_pool():
    c = TreeCase([14], [star(33)], stale="normal").to_device()
    c.tables()
    c.tree.path[:2] = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
    c.tree.n_kept.fill_(2)
    c.L.block_table[0, 2] = 10 ** 6
    before = c.dk.clone()
    pcf.tree_keep(c.L, c.tree, [c.dk], [c.dv])
    raises(BOUNDS)
    assert torch.equal(c.dk, before)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("shape", [dict(hq=8, hkv=2, d=64, theta=1e4), dict(hq=32, hkv=8, d=128, theta=5e5)])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_drafted_trees(shape, captured):
    """Many steps of two layers: every step's trees attend over what the steps before kept; each result, the
    branch, the lengths, the pages in use and every kept key and value against the tokens' own record."""
    hq, hkv, d, theta = (shape[k] for k in ("hq", "hkv", "d", "theta"))
    layers, n, nodes, max_pos, n_phys, steps = 2, 3, 12, 400, 40, 12
    rng = np.random.default_rng(hq)
    g = torch.Generator().manual_seed(hq)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    L = pcf.ChunkLayout(n, hq, hkv, d, n_phys, max_pos, max_pages=12, max_rows=n * nodes, max_chunk=nodes)
    T = pcf.DraftTree(L)
    free, head, seq = torch.randperm(n_phys, generator=g).to(torch.int32).cuda(), i32([0]), i32([0] * n)
    new, parent, draft, choice = i32([0] * n), i32([0] * n * nodes), i32([0] * n * nodes), i32([0] * n * nodes)
    kp = [torch.full((n_phys, hkv, PAGE, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    vp = [torch.full_like(kp[0], float("nan")) for _ in range(layers)]
    rows = lambda h: [torch.zeros((n * nodes, h, d), dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    q, k, v, out = rows(hq), rows(hkv), rows(hkv), rows(hq)
    rope = pcf.rope_table(d, theta, max_pos).cuda()
    ws = torch.empty(max(16, T.attention_workspace_bytes()), dtype=torch.uint8, device="cuda")

    def step():
        pcf.chunk_tables(L, seq, new, free, head, seq, head)
        pcf.tree_tables(L, T, parent)
        for l in range(layers):
            pcf.append_kv(L, k[l], v[l], kp[l], vp[l])
            pcf.tree_attention(L, T, q[l], kp[l], vp[l], rope, out[l], ws)
        pcf.tree_accept(L, T, parent, draft, choice, free, seq, head)
        pcf.tree_keep(L, T, kp, vp)

    if captured:
        step()                                     # (no new tokens: loads the kernels)
        pcf.check_device_error()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    held = [[[np.zeros((0, hkv, d)) for _ in range(2)] for _ in range(layers)] for _ in range(n)]
    for i in range(steps):
        sizes = [int(x) for x in rng.integers(0 if i else 1, nodes + 1, n)]
        parents = trees(sizes, int(rng.integers(1 << 30)), 4)
        total = sum(sizes)
        dr, ch = rng.integers(0, 3, n * nodes), rng.integers(0, 3, n * nodes)
        flat = [p for t in parents for p in t]
        new.copy_(i32(sizes)), draft.copy_(i32(dr.tolist())), choice.copy_(i32(ch.tolist()))
        parent.copy_(i32(flat + [0] * (n * nodes - total)))
        host = [[bf16(g, n * nodes, h, d) for h in (hq, hkv, hkv)] for _ in range(layers)]
        for l in range(layers):
            for dst, src in zip((q[l], k[l], v[l]), host[l]):
                dst.copy_(src)
        graph.replay() if captured else step()
        pcf.check_device_error()
        base = 0
        for b in range(n):
            m = sizes[b]
            kept, said = tree.branch(parents[b], dr[base: base + m], ch[base: base + m])
            s = len(held[b][0][0])
            pos, bits = tree.tables([parents[b]], [s], 1)
            seen = np.ones((m, s + m), dtype=bool)
            seen[:, s:] = (bits >> np.arange(m, dtype=np.uint32)) & 1
            where = np.concatenate([np.arange(s), pos])
            for l in range(layers):
                hq_, hk, hv = (x[base: base + m].double().numpy() for x in host[l])
                K, V = np.concatenate([held[b][l][0], hk]), np.concatenate([held[b][l][1], hv])
                o, mean_abs, score_abs = chunk.attention(hq_, pos, K, V, where, seen, theta)
                got = out[l][base: base + m].float().cpu().double().numpy()
                assert np.all(np.abs(got - o) <= chunk.attention_bound(o, mean_abs, score_abs)), (i, b, l)
                held[b][l] = [np.concatenate([old, x[kept]]) for old, x in zip(held[b][l], (hk, hv))]
            assert T.path[base: base + m].tolist() == kept + [-1] * (m - len(kept))
            assert T.n_kept[b].item() == len(kept) and T.next_token[b].item() == said
            s = len(held[b][0][0])
            assert seq[b].item() == s
            pages = L.block_table[b, : -(-s // PAGE)].long()
            for l in range(layers):
                for pool, mine in zip((kp[l], vp[l]), held[b][l]):
                    got = pool[pages].transpose(1, 2).reshape(-1, hkv, d)[:s].double().cpu().numpy()
                    assert np.array_equal(got, mine), (i, b, l)
            base += m
        # every page is held once or free once
        used = [p for b in range(n) for p in L.block_table[b, : -(-seq[b].item() // PAGE)].tolist()]
        assert head.item() == len(used) and sorted(used + free[head.item():].tolist()) == list(range(n_phys)), i


def test_two_captured_graphs_share_a_workspace_in_order():
    a = TreeCase([900, 20], trees([5, 40], 1), hq=32, hkv=8, d=128, seed=1).to_device()
    b = TreeCase([30, 500], trees([70, 1], 2), hq=32, hkv=8, d=128, seed=2).to_device()
    a.ws = b.ws = torch.empty(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    graphs = []
    for c in (a, b):
        c.step()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.tables()
            c.append()
            c.attend()
            c.accept()
        graphs.append(gr)
    a.out.fill_(3.0), b.out.fill_(3.0)
    for _ in range(4):
        for gr in graphs:
            gr.replay()
    pcf.check_device_error()
    for c in (a, b):
        c.check(c.out.float().cpu().double().numpy(), rows=6)
        check_accepted(c)
