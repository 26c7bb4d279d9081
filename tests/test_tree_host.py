"""CPU tests of the calls that check drafted trees: refusals before any launch, sizes, the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf
from oracle import chunk, tree
from position_independent_kv_critical_gb300 import _lib

from test_chunk_host import BUF, INVALID, NO_DEVICE, P, TOO_SMALL, UNSUPPORTED, dims
from tree_util import chain, random_tree, star


@pytest.mark.parametrize("kw,status", [
    (dict(n_reqs=0), INVALID), (dict(max_rows=0), INVALID), (dict(max_chunk=21), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(n_q_heads=6), UNSUPPORTED), (dict(max_rows=257, max_chunk=257), UNSUPPORTED),
    (dict(max_rows=1 << 22, max_chunk=2, n_q_heads=512, n_kv_heads=512), INVALID)])     # rows of the rotated queries
def test_dims_out_of_range_are_refused(lib, kw, status):
    n, size = ctypes.c_int64(0), ctypes.c_size_t(0)
    d = ctypes.byref(dims(**kw))
    assert lib.pcf_tree_plan_words(d, ctypes.byref(n)) == status
    assert lib.pcf_tree_attention_workspace_bytes(d, ctypes.byref(size)) == status
    assert lib.pcf_tree_tables(d, *[None] * 6) == status
    assert lib.pcf_tree_attention(d, None, None, 0, *[None] * 10, 0, None) == status
    assert lib.pcf_tree_accept(d, *[None] * 8, 0, *[None] * 6) == status
    assert lib.pcf_tree_keep(d, *[None] * 4, 1, None, None, None) == status


def test_sizes(lib):
    n, size = ctypes.c_int64(0), ctypes.c_size_t(0)
    for kw in (dict(), dict(max_rows=256, max_chunk=256), dict(n_sms=1), dict(n_reqs=4096)):
        d = ctypes.byref(dims(**kw))
        assert lib.pcf_tree_plan_words(d, ctypes.byref(n)) == 0 and n.value > 4 * dims(**kw).n_reqs
        assert lib.pcf_tree_attention_workspace_bytes(d, ctypes.byref(size)) == 0 and size.value >= 0
    assert lib.pcf_tree_plan_words(None, ctypes.byref(n)) == INVALID
    assert lib.pcf_tree_plan_words(ctypes.byref(dims()), None) == INVALID
    assert lib.pcf_tree_attention_workspace_bytes(ctypes.byref(dims()), None) == INVALID


def test_tables_refuse_null_and_misaligned_pointers(lib):
    d = ctypes.byref(dims())
    args = [P] * 5 + [None]
    for i in range(5):
        for bad_value in (None, P + 2):
            bad = list(args)
            bad[i] = bad_value
            assert lib.pcf_tree_tables(d, *bad) == INVALID, (i, bad_value)
    bad = list(args)
    bad[4] = P + 4                                         # the plan: 16 bytes
    assert lib.pcf_tree_tables(d, *bad) == INVALID
    if not torch.cuda.is_available():
        assert lib.pcf_tree_tables(d, *args) == NO_DEVICE


def test_attention_refuses_bad_pointers_strides_overlap_and_workspace(lib):
    d = ctypes.byref(dims())
    size = ctypes.c_size_t(0)
    assert lib.pcf_tree_attention_workspace_bytes(d, ctypes.byref(size)) == 0
    Q, O = P, P + 8 * (1 << 15)
    #       plan q  stride k  v  table pos excl row_pos seen rope out ws bytes       stream
    args = [P, Q, 8 * 64, P, P, P, P, None, P, P, P, O, P, size.value, None]
    for i in (0, 1, 3, 4, 5, 6, 8, 9, 10, 11, 12):
        bad = list(args)
        bad[i] = None
        assert lib.pcf_tree_attention(d, *bad) == INVALID, i
        bad[i] = (O if i == 11 else P) + (2 if i in (5, 6, 8, 9) else 8)
        assert lib.pcf_tree_attention(d, *bad) == INVALID, i
    for stride in (8 * 64 - 8, 8 * 64 + 4, 0, -512):
        bad = list(args)
        bad[2] = stride
        assert lib.pcf_tree_attention(d, *bad) == INVALID, stride
    bad = list(args)
    bad[7] = P + 1
    assert lib.pcf_tree_attention(d, *bad) == INVALID
    for at in (P, P + 1024, P + 20 * 1024 - 16):           # out overlaps q
        bad = list(args)
        bad[11] = at
        assert lib.pcf_tree_attention(d, *bad) == INVALID
    if size.value:
        bad = list(args)
        bad[13] = size.value - 1
        assert lib.pcf_tree_attention(d, *bad) == TOO_SMALL
    if not torch.cuda.is_available():
        assert lib.pcf_tree_attention(d, *args) == NO_DEVICE


def test_accept_refuses_null_and_misaligned_pointers(lib):
    d = ctypes.byref(dims())
    #       chunk tree parent draft choice root table free n path kept next seq head stream
    args = [P, P, P, P, P, None, P, P, 5, P, P, P, P, P, None]
    for i in (0, 1, 2, 3, 4, 6, 7, 9, 10, 11, 12, 13):
        for bad_value in (None, P + 2):
            bad = list(args)
            bad[i] = bad_value
            assert lib.pcf_tree_accept(d, *bad) == INVALID, (i, bad_value)
    for i, bad_value in ((5, P + 2), (1, P + 4), (8, -1)):
        bad = list(args)
        bad[i] = bad_value
        assert lib.pcf_tree_accept(d, *bad) == INVALID, (i, bad_value)
    if not torch.cuda.is_available():
        assert lib.pcf_tree_accept(d, *args) == NO_DEVICE
        assert lib.pcf_tree_accept(d, *args[:7], None, 0, *args[9:]) == NO_DEVICE       # an empty list


def test_keep_refuses_bad_pointers_and_numbers_of_layers(lib):
    d = ctypes.byref(dims())
    size = 40 * 2 * 16 * 64 * 2                            # of a pool of these dims
    pools = [(ctypes.c_void_p * 2)(*[P + size * (2 * i + j) for i in range(2)]) for j in range(2)]
    args = [P, P, P, P, 2, *pools, None]
    for i in (0, 1, 2, 3, 5, 6):
        bad = list(args)
        bad[i] = None
        assert lib.pcf_tree_keep(d, *bad) == INVALID, i
        if i < 4:
            bad[i] = P + (4 if i == 0 else 2)
            assert lib.pcf_tree_keep(d, *bad) == INVALID, i
    for n in (0, -1, 4097):
        bad = list(args)
        bad[4] = n
        assert lib.pcf_tree_keep(d, *bad) == INVALID
    for wrong in (None, P + 8):
        for which in (5, 6):
            bad = list(args)
            bad[which] = (ctypes.c_void_p * 2)(args[which][0], wrong)
            assert lib.pcf_tree_keep(d, *bad) == INVALID
    for k, v in (((0, 2), (1, 2)), ((0, 0), (1, 2)), ((0, 1), (0, 3)), ((0, 1.5), (2, 4))):       # pools that overlap
        bad = list(args)
        bad[5], bad[6] = ((ctypes.c_void_p * 2)(*[P + int(size * x) for x in w]) for w in (k, v))
        assert lib.pcf_tree_keep(d, *bad) == INVALID, (k, v)
    if not torch.cuda.is_available():
        assert lib.pcf_tree_keep(d, *args) == NO_DEVICE


def test_binding_refuses_tensors_of_other_shapes_types_and_layouts():
    new = lambda **kw: pcf.ChunkLayout(3, 8, 2, 64, 40, 512, **{**dict(max_pages=8, max_rows=20, max_chunk=9, device="cpu"), **kw})
    L = new()
    T = pcf.DraftTree(L)
    assert T.row_pos.shape == (20,) and T.seen.shape == (20, 1) and pcf.DraftTree(new(max_rows=40, max_chunk=33)).seen.shape == (40, 2)
    with pytest.raises(pcf.PcfError, match="UNSUPPORTED"):
        pcf.DraftTree(new(max_rows=300, max_chunk=257))
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError, match="another layout"):
        pcf.tree_tables(new(), T, i32(20))
    for bad in (i32(19), i32(20).long(), i32(40)[::2]):
        with pytest.raises(ValueError, match="parent"):
            pcf.tree_tables(L, T, bad)
    pool = torch.zeros((40, 2, 16, 64), dtype=torch.bfloat16)
    q = torch.zeros((20, 8, 64), dtype=torch.bfloat16)
    rope, ws = torch.zeros((512, 32, 2)), torch.zeros(64, dtype=torch.uint8)
    ok = dict(q=q, k_pool=pool, v_pool=pool, rope=rope, out=torch.zeros_like(q), ws=ws)
    for name, bad in (("q", q[:19]), ("q", q.float()), ("k_pool", pool[:39]), ("v_pool", pool.float()), ("rope", rope[:511]),
                      ("out", q[:19]), ("excl", torch.zeros((3, 7), dtype=torch.int16)), ("ws", torch.zeros(64)[::2])):
        with pytest.raises(ValueError, match=name):
            pcf.tree_attention(L, T, **{**ok, name: bad})
    ok = dict(parent=i32(20), draft=i32(20), choice=i32(20), free_pages=i32(5), seq_len_out=i32(3), free_head_out=i32(1))
    for name, bad in (("parent", i32(19)), ("draft", i32(21)), ("choice", i32(20).float()), ("free_pages", i32(10)[::2]),
                      ("seq_len_out", i32(2)), ("free_head_out", i32(2)), ("root_choice", i32(20))):
        with pytest.raises(ValueError, match=name):
            pcf.tree_accept(L, T, **{**ok, name: bad})
    for k, v in (([pool], [pool, pool]), ([], []), ([pool[:39]], [pool]), ([pool], [pool.float()])):
        with pytest.raises(ValueError, match="pools"):
            pcf.tree_keep(L, T, k, v)
    with pytest.raises(AttributeError):
        T.row_pos = i32(20)
    for call in (lambda: pcf.tree_tables(L, T, i32(20)), lambda: pcf.tree_accept(L, T, **ok),
                 lambda: pcf.tree_keep(L, T, [pool], [pool.clone()])):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


# ------------------------------------------------------------------ the oracle itself
@pytest.mark.parametrize("parent", [[-1], chain(9), star(9), [-1, 0, 0, 1, 1, 2, 5, 0, -1, 8]])
def test_every_line_is_a_request_of_its_own(parent):
    """A node's result is that of the last token of a request that holds the same tokens and its line."""
    rng = np.random.default_rng(len(parent))
    s, hq, hkv, d, theta, first = 21, 4, 2, 64, 1e4, 9
    n = s + len(parent)
    q = rng.standard_normal((len(parent), hq, d))
    k, v = rng.standard_normal((n, hkv, d)), rng.standard_normal((n, hkv, d))
    pos, bits = tree.tables([parent], [first + s], 1)
    where = np.concatenate([first + np.arange(s), pos])
    seen = np.ones((len(parent), n), dtype=bool)
    seen[:, s:] = (bits >> np.arange(len(parent), dtype=np.uint32)) & 1
    out, _, _ = chunk.attention(q, pos, k, v, where, seen, theta)
    for t, line in enumerate(tree.lines(parent)):
        mine = list(range(s)) + [s + u for u in line]
        at = first + np.arange(len(mine))
        alone, _, _ = chunk.attention(q[t: t + 1], at[-1:], k[mine], v[mine], at, np.ones((1, len(mine)), dtype=bool), theta)
        assert np.allclose(out[t], alone[0], atol=1e-12)


def test_bits_and_positions_of_known_trees():
    pos, bits = tree.tables([chain(3), star(3), []], [5, 100, 7], 1)
    assert pos.tolist() == [5, 6, 7, 100, 101, 101] and bits[:, 0].tolist() == [1, 3, 7, 1, 3, 5]
    pos, bits = tree.tables([chain(70)], [0], 3)
    assert bits[69].tolist() == [0xFFFFFFFF, 0xFFFFFFFF, 63] and pos[69] == 69


def test_branches():
    parent, draft = [-1, 0, 0, 1, 2, 2, -1], [7, 1, 2, 3, 4, 4, 8]
    assert tree.branch(parent, draft, [2, 0, 4, 0, 9, 6, 0]) == ([0, 2, 4], 9)      # of two equal siblings the first
    assert tree.branch(parent, draft, [5, 0, 0, 0, 0, 0, 0]) == ([0], 5)
    assert tree.branch(parent, draft, [5, 0, 0, 0, 0, 0, 3], root=8) == ([6], 3)
    assert tree.branch(parent, draft, [5, 0, 0, 0, 0, 0, 3], root=1) == ([], 1)
    assert tree.branch([], [], []) == ([], -1) and tree.branch([], [], [], root=4) == ([], 4)


def test_pages_go_back_in_order():
    table = [[9, 4, 5, 6], [1, 2, 0, 0], [3, 0, 0, 0]]
    #         16 held + 33 nodes take 4, 5, 6; 10 + 7 take 2; 0 + 2 take 3
    parents = [chain(33), star(7), chain(2)]
    draft, choice = list(range(33)) + [50] * 7 + [1, 2], [1, 2, 3] + [0] * 37 + [2, 9]
    path, kept, token, length, free, head = tree.accept([16, 10, 0], parents, draft, choice, None, table,
                                                       [99, 4, 5, 6, 2, 3, 77], 1, 5)
    assert kept == [4, 1, 2] and token == [0, 0, 9] and length == [20, 11, 2]
    assert path[:5] == [0, 1, 2, 3, -1] and path[33:35] == [0, -1] and path[40:] == [0, 1]
    assert free == [99, 4, 5, 5, 6, 2, 77] and head == 3       # 4 (and 3, behind) stay taken


def test_kept_entries_move_together():
    pool = np.arange(4 * 16).reshape(4, 1, 16).astype(float)
    out = tree.keep(pool, [14], [0], [0, 2, 3, 20], [4], [[3, 0, 1, 2]])
    assert out[3, 0].tolist() == [48.0 + i for i in range(16)][:15] + [0.0]
    assert out[0, 0].tolist()[:2] == [1.0, 16.0 + 2.0] and out[1, 0].tolist() == pool[1, 0].tolist()


def test_random_trees_have_parents_first():
    rng = np.random.default_rng(0)
    for n in (1, 2, 40, 256):
        for width in (None, 1, 7):
            assert all(-1 <= p < t for t, p in enumerate(random_tree(n, rng, width, roots=True)))
