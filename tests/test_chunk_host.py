"""CPU tests of the calls that continue a request: refusals before any launch, sizes, the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import position_independent_kv_critical_gb300 as pcf
from oracle import chunk, method
from oracle.rope import rotate
from position_independent_kv_critical_gb300 import _lib

INVALID, UNSUPPORTED, TOO_SMALL, NO_DEVICE = -1, -2, -5, -7


def dims(**kw):
    base = dict(n_reqs=3, max_pages=8, max_rows=20, max_chunk=9, max_total_pages=24, n_q_heads=8, n_kv_heads=2,
                head_dim=64, n_phys_pages=40, max_pos=512, n_sms=0)
    return _lib.ChunkDims(**{**base, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(n_reqs=0), INVALID), (dict(n_reqs=4097), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pages=65537), INVALID), (dict(max_rows=0), INVALID), (dict(max_rows=(1 << 22) + 1), INVALID),
    (dict(max_chunk=0), INVALID), (dict(max_chunk=21), INVALID), (dict(max_total_pages=0), INVALID),
    (dict(max_total_pages=(1 << 26) + 1), INVALID), (dict(n_q_heads=9), INVALID), (dict(n_q_heads=0), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(n_q_heads=2048), INVALID), (dict(n_phys_pages=0), INVALID),
    (dict(n_phys_pages=1 << 26), INVALID), (dict(max_pos=15), INVALID), (dict(max_pos=(1 << 20) + 1), INVALID),
    (dict(n_sms=4097), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(n_q_heads=6), UNSUPPORTED)])
def test_dims_out_of_range_are_refused(lib, kw, status):
    n, size = ctypes.c_int64(0), ctypes.c_size_t(0)
    d = dims(**kw)
    assert lib.pcf_chunk_plan_words(ctypes.byref(d), ctypes.byref(n)) == status
    assert lib.pcf_chunk_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(size)) == status
    assert lib.pcf_chunk_tables(ctypes.byref(d), *[None] * 4, 0, *[None] * 10) == status
    assert lib.pcf_append_kv(ctypes.byref(d), None, 0, None, 0, *[None] * 7) == status
    assert lib.pcf_chunk_attention(ctypes.byref(d), None, None, 0, *[None] * 9, 0, None) == status


def test_null_dims_and_null_results_are_refused(lib):
    n, size = ctypes.c_int64(0), ctypes.c_size_t(0)
    d = dims()
    assert lib.pcf_chunk_plan_words(None, ctypes.byref(n)) == INVALID
    assert lib.pcf_chunk_plan_words(ctypes.byref(d), None) == INVALID
    assert lib.pcf_chunk_attention_workspace_bytes(ctypes.byref(d), None) == INVALID
    assert lib.pcf_chunk_plan_words(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.pcf_chunk_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(size)) == 0


# host buffers stand in for device ones: every call below is refused before it could launch
BUF = torch.zeros(1 << 16, dtype=torch.int64)
P = BUF.data_ptr()


def test_tables_refuse_null_and_misaligned_pointers(lib):
    d = dims()
    args = [P] * 4 + [5] + [P] * 10
    for i in (0, 1, 3, 5, 6, 7, 8, 9, 10, 11, 12, 13):
        bad = list(args)
        bad[i] = None
        assert lib.pcf_chunk_tables(ctypes.byref(d), *bad) == INVALID, i
        bad[i] = P + 2
        assert lib.pcf_chunk_tables(ctypes.byref(d), *bad) == INVALID, i
    bad = list(args)
    bad[4] = -1
    assert lib.pcf_chunk_tables(ctypes.byref(d), *bad) == INVALID


def test_append_refuses_bad_pointers_and_strides(lib):
    d = dims()
    args = [P, 128, P, 128] + [P] * 6 + [None]
    for i in (0, 2, 4, 8, 9):
        bad = list(args)
        bad[i] = None
        assert lib.pcf_append_kv(ctypes.byref(d), *bad) == INVALID, i
    for i in (0, 2, 7, 8, 9):
        bad = list(args)
        bad[i] = P + 8
        assert lib.pcf_append_kv(ctypes.byref(d), *bad) == INVALID, i
    for i in (1, 3):
        for stride in (127, 120, 132, 0, -128):
            bad = list(args)
            bad[i] = stride
            assert lib.pcf_append_kv(ctypes.byref(d), *bad) == INVALID, (i, stride)
    for i in (5, 7):        # row_pos needs slot_pos and rope
        bad = list(args)
        bad[i] = None
        assert lib.pcf_append_kv(ctypes.byref(d), *bad) == INVALID, i


def test_attention_refuses_bad_pointers_strides_and_workspaces(lib):
    d = dims()
    size = ctypes.c_size_t(0)
    lib.pcf_chunk_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(size))
    #       plan q  stride   k  v  table pos excl row_pos rope out ws  bytes       stream
    out = P + 8 * (1 << 15)
    args = [P, P, 512, P, P, P, P, P, P, P, out, P, size.value, None]
    for i in (0, 1, 3, 4, 5, 6, 8, 9, 10, 11):
        bad = list(args)
        bad[i] = None
        assert lib.pcf_chunk_attention(ctypes.byref(d), *bad) == INVALID, i
    for i, off in ((0, 2), (1, 8), (3, 8), (4, 8), (5, 2), (6, 2), (7, 1), (8, 2), (9, 8), (10, 8), (11, 8)):
        bad = list(args)
        bad[i] = args[i] + off
        assert lib.pcf_chunk_attention(ctypes.byref(d), *bad) == INVALID, i
    for stride in (511, 504, 516, 0):
        bad = list(args)
        bad[2] = stride
        assert lib.pcf_chunk_attention(ctypes.byref(d), *bad) == INVALID
    for at in (P, P + 1024, P + 20 * 1024 - 16):          # out overlaps q
        bad = list(args)
        bad[10] = at
        assert lib.pcf_chunk_attention(ctypes.byref(d), *bad) == INVALID
    if size.value:
        bad = list(args)
        bad[12] = size.value - 1
        assert lib.pcf_chunk_attention(ctypes.byref(d), *bad) == TOO_SMALL
    if not torch.cuda.is_available():
        assert lib.pcf_chunk_attention(ctypes.byref(d), *args) == NO_DEVICE


def test_binding_refuses_tensors_of_other_shapes_types_and_strides():
    L = pcf.ChunkLayout(3, 8, 2, 64, 40, 512, max_pages=8, max_rows=20, max_chunk=9, device="cpu")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    ok = dict(seq_len=i32(3), new_len=i32(3), free_pages=i32(5), free_head=i32(1), seq_len_out=i32(3),
              free_head_out=i32(1))
    for name, bad in (("seq_len", i32(4)), ("new_len", i32(3).long()), ("seq_len_out", i32(2)),
                      ("free_head", i32(2)), ("free_pages", i32(10)[::2])):
        with pytest.raises(ValueError, match=name):
            pcf.chunk_tables(L, **{**ok, name: bad})
    pool = torch.zeros((40, 2, 16, 64), dtype=torch.bfloat16)
    kv = torch.zeros((20, 2, 64), dtype=torch.bfloat16)
    wide = torch.zeros((20, 2, 128), dtype=torch.bfloat16)
    for bad in (kv[:19], kv.float(), wide[:, :, ::2], wide[:, :, :64], kv[:1].expand(20, 2, 64)):
        with pytest.raises(ValueError, match="k_new"):
            pcf.append_kv(L, bad, kv, pool, pool)
    with pytest.raises(ValueError, match="v_pool"):
        pcf.append_kv(L, kv, kv, pool, pool[:39])
    q = torch.zeros((20, 8, 64), dtype=torch.bfloat16)
    rope, ws = torch.zeros((512, 32, 2)), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="rope"):
        pcf.chunk_attention(L, q, pool, pool, rope[:511], q, ws)
    with pytest.raises(ValueError, match="excl"):
        pcf.chunk_attention(L, q, pool, pool, rope, q, ws, excl=torch.zeros((3, 7), dtype=torch.int16))
    with pytest.raises(ValueError, match="out"):
        pcf.chunk_attention(L, q, pool, pool, rope, q[:19], ws)
    # host tensors of the right kinds
    with pytest.raises(ValueError, match="not on a GPU"):
        pcf.chunk_tables(L, **ok)
    with pytest.raises(ValueError, match="not on a GPU"):
        pcf.append_kv(L, kv, kv, pool, pool)
    with pytest.raises(ValueError, match="not on a GPU"):
        pcf.chunk_attention(L, q, pool, pool, rope, torch.zeros_like(q), ws)


def test_tables_are_replaced_only_by_tables_of_the_same_kind():
    L = pcf.ChunkLayout(3, 8, 2, 64, 40, 512, max_pages=8, max_rows=20, max_chunk=9, device="cpu")
    other = torch.zeros((3, 8), dtype=torch.int32)
    L.block_table = other
    assert L.block_table is other
    for bad in (other[:2], other.long(), torch.zeros((8, 3), dtype=torch.int32).t(), torch.zeros(24, dtype=torch.int32)):
        with pytest.raises(ValueError, match="block_table"):
            L.block_table = bad
    with pytest.raises(ValueError, match="plan"):
        L.plan = L.plan[:-1]


def test_layout_from_a_fused_batch_lists_its_spans():
    from workload import small_custom_batch
    b = small_custom_batch([(0, 3, 7, 5), (20, 2, 60, 1)], 2, hq=8, hkv=2, d=64, n_phys_pages=40,
                           extra_requests=[([(3, 17, 100, 40)], 3, 400), ([], 4, 10)])
    lay = pcf.Layout(b.requests, 8, 2, 64, 40, 512, device="cpu")
    excl = torch.arange(lay.total_pages, dtype=torch.int16) + 1
    L, words = pcf.ChunkLayout.from_layout(lay, max_pages=20, max_rows=60, max_chunk=50, max_pos=512, excl=excl,
                                           device="cpu")
    assert L.block_table[0, :6].tolist() == [0, 1, 2, 20, 21, 0]
    assert L.page_pos[0, :6].tolist() == [7, 23, 39, 60, 76, 0]
    assert L.block_table[1, :18].tolist() == list(range(3, 20)) + [0]
    assert words[0].tolist() == [1, 2, 3, 4, 5] + [0] * 15
    assert words[1].tolist() == list(range(6, 23)) + [0] * 3 and not words[2].any()
    with pytest.raises(ValueError, match="max_pages"):
        pcf.ChunkLayout.from_layout(lay, max_pages=16, max_rows=60, max_chunk=50, max_pos=512, device="cpu")


# ------------------------------------------------------------------ the oracle itself
def test_oracle_chunk_equals_full_prefill():
    """Attending chunk by chunk over pages is the same causal prefill as all tokens at once."""
    rng = np.random.default_rng(3)
    n, hq, hkv, d, theta = 45, 4, 2, 64, 1e4
    q, k, v = rng.standard_normal((n, hq, d)), rng.standard_normal((n, hkv, d)), rng.standard_normal((n, hkv, d))
    whole = method.full_prefill(q, k, v, np.arange(n) + 9, theta)
    pool_k, pool_v = np.full((8, hkv, 16, d), np.nan), np.full((8, hkv, 16, d), np.nan)
    bt, pp = np.zeros((1, 4), dtype=int), np.zeros((1, 4), dtype=int)
    free, head, seq = [5, 2, 7, 0], 0, 0
    for new in (1, 15, 1, 20, 8):
        bt, pp, slots, where, base, head = chunk.tables([seq], [new], free, head, bt, pp, [9 + seq])
        assert base.tolist() == [0, new] and where.tolist() == list(range(9 + seq, 9 + seq + new))
        pool_k[slots // 16, :, slots % 16], pool_v[slots // 16, :, slots % 16] = k[seq: seq + new], v[seq: seq + new]
        m = seq + new
        pages = bt[0, : -(-m // 16)]
        pos = (pp[0, : len(pages), None] + np.arange(16)).reshape(-1)[:m]
        seen = np.arange(m)[None] <= seq + np.arange(new)[:, None]
        out, _, _ = chunk.attention(q[seq:m], where, chunk.gather(pool_k, pages, m), chunk.gather(pool_v, pages, m), pos,
                                    seen, theta)
        assert np.allclose(out, whole[seq:m], atol=1e-12)
        seq = m


def test_oracle_key_stored_for_another_slot_turns_back():
    rng = np.random.default_rng(4)
    k = rng.standard_normal((6, 2, 64))
    at, slot = np.array([3, 90, 41, 7, 100, 55]), np.array([80, 81, 82, 83, 84, 85])
    assert np.allclose(rotate(chunk.appended(k, slot, at, 1e4), slot, 1e4), rotate(k, at, 1e4), atol=1e-12)
