"""A batch of requests that go on from a page pool: seeded inputs, the calls, the oracle's answer."""
from __future__ import annotations

import numpy as np
import torch

import position_independent_kv_critical_gb300 as pcf
from oracle import chunk

PAGE = 16


def bf16(gen, *shape):
    return torch.randn(shape, generator=gen, dtype=torch.float32).to(torch.bfloat16)


class ChunkCase:
    """Requests with seq[b] tokens held and new[b] to come.  Pages are drawn in random order from one
    pool; request b starts at position pos0 + 37 b.  ``stale``: what fills every slot that holds no token
    ("nan": NaN, otherwise normal draws)."""

    def __init__(self, seq, new, hq=8, hkv=2, d=64, theta=1e4, seed=1, pos0=5, spare_rows=0, extra_pages=3,
                 max_pages=None, max_chunk=None, next_pos=True, n_phys=None, stale="nan", device="cuda"):
        self.seq, self.new = list(seq), list(new)
        self.hq, self.hkv, self.d, self.theta, self.n = hq, hkv, d, theta, len(seq)
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        held = [-(-s // PAGE) for s in seq]
        after = [-(-(s + m) // PAGE) for s, m in zip(seq, new)]
        self.rows = sum(new)
        self.max_rows = max(1, self.rows + spare_rows)
        self.max_pages = max(1, max(after)) if max_pages is None else max_pages
        self.n_phys = sum(after) + extra_pages if n_phys is None else n_phys
        self.max_pos = pos0 + 37 * self.n + max(s + m for s, m in zip(seq, new)) + 2 * PAGE
        order = rng.permutation(self.n_phys)
        self.table = np.zeros((self.n, self.max_pages), dtype=np.int32)
        self.page_pos = np.zeros_like(self.table)
        at = 0
        for b in range(self.n):
            self.table[b, : held[b]] = order[at: at + held[b]]
            self.page_pos[b, : held[b]] = pos0 + 37 * b + PAGE * np.arange(held[b])
            at += held[b]
        self.free = order[at:].astype(np.int32)
        self.next_pos = (np.array([pos0 + 37 * b + s for b, s in enumerate(seq)], dtype=np.int32) if next_pos else None)
        (self.bt, self.pp, self.slots, self.where, self.base, self.head) = chunk.tables(
            self.seq, self.new, self.free, 0, self.table, self.page_pos, self.next_pos)
        self.k_pool = bf16(g, self.n_phys, hkv, PAGE, d)
        self.v_pool = bf16(g, self.n_phys, hkv, PAGE, d)
        self.q = bf16(g, self.max_rows, hq, d)
        self.k_new, self.v_new = bf16(g, self.max_rows, hkv, d), bf16(g, self.max_rows, hkv, d)
        if stale == "nan":      # every slot that holds no token
            full = torch.zeros((self.n_phys, PAGE), dtype=torch.bool)
            for b in range(self.n):
                for j in range(self.seq[b]):
                    full[self.table[b, j // PAGE], j % PAGE] = True
            for t in (self.k_pool, self.v_pool):
                t.masked_fill_(~full[:, None, :, None], float("nan"))
        self.excl = None
        self.max_chunk = max(1, max(new)) if max_chunk is None else max_chunk

    # ---- device side
    def layout(self, device="cuda", **kw):
        L = pcf.ChunkLayout(self.n, self.hq, self.hkv, self.d, self.n_phys, self.max_pos, max_pages=self.max_pages,
                            max_rows=self.max_rows, max_chunk=self.max_chunk, device=device, **kw)
        L.block_table.copy_(torch.from_numpy(self.table))
        L.page_pos.copy_(torch.from_numpy(self.page_pos))
        return L

    def to_device(self):
        i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()
        self.L = self.layout()
        self.d_seq, self.d_new, self.d_free = i32(self.seq), i32(self.new), i32(self.free)
        self.d_next = None if self.next_pos is None else i32(self.next_pos)
        self.d_head = i32([0])
        self.d_seq_out, self.d_head_out = torch.full_like(self.d_seq, -7), torch.full_like(self.d_head, -7)
        self.dk, self.dv = self.k_pool.cuda(), self.v_pool.cuda()
        self.dq, self.dkn, self.dvn = self.q.cuda(), self.k_new.cuda(), self.v_new.cuda()
        self.rope = pcf.rope_table(self.d, self.theta, self.max_pos).cuda()
        self.out = torch.full((self.max_rows, self.hq, self.d), 3.0, dtype=torch.bfloat16, device="cuda")
        self.ws = torch.empty(max(16, self.L.attention_workspace_bytes()), dtype=torch.uint8, device="cuda")
        self.d_excl = None if self.excl is None else torch.from_numpy(self.excl.view(np.int16)).cuda()
        return self

    def tables(self, **kw):
        pcf.chunk_tables(self.L, self.d_seq, self.d_new, self.d_free, self.d_head, self.d_seq_out, self.d_head_out,
                         next_pos=self.d_next, **kw)

    def append(self, **kw):
        pcf.append_kv(self.L, self.dkn, self.dvn, self.dk, self.dv, rope=self.rope, **kw)

    def attend(self, **kw):
        pcf.chunk_attention(self.L, self.dq, self.dk, self.dv, self.rope, self.out, self.ws, excl=self.d_excl, **kw)

    def step(self):
        self.tables()
        self.append()
        self.attend()
        pcf.check_device_error()
        return self.out.float().cpu().double().numpy()

    # ---- oracle side: the pool after the append, then every request (or some of its rows)
    def oracle(self, b, rows=None):
        n = self.seq[b] + self.new[b]
        k, v = self.k_pool.double().numpy().copy(), self.v_pool.double().numpy().copy()
        sl = slice(self.base[b], self.base[b + 1])
        page, r = self.slots[sl] // PAGE, self.slots[sl] % PAGE
        k[page, :, r] = self.k_new[sl].double().numpy()
        v[page, :, r] = self.v_new[sl].double().numpy()
        pages = self.bt[b, : -(-n // PAGE)]
        pos = (self.pp[b, : len(pages), None] + np.arange(PAGE)).reshape(-1)[:n]
        K, V = chunk.gather(k, pages, n), chunk.gather(v, pages, n)
        seen = np.arange(n)[None] <= self.seq[b] + np.arange(self.new[b])[:, None]
        if self.excl is not None:
            gone = ((self.excl[b, : len(pages), None].astype(np.int64) >> np.arange(PAGE)) & 1).reshape(-1)[:n]
            seen = seen & (gone == 0)[None]
        K = np.where(seen.any(axis=0)[:, None, None], K, 0.0)
        t = np.arange(self.new[b]) if rows is None else np.asarray(rows)
        q = self.q[sl].double().numpy()[t]
        return t, chunk.attention(q, self.where[sl][t], K, V, pos, seen[t], self.theta)

    def check(self, got, rows=None):
        assert np.all(got[self.rows:] == 3.0), "rows behind the last one were written"
        for b in range(self.n):
            if self.new[b] == 0:
                continue
            pick = None if rows is None else sorted({0, self.new[b] - 1, *np.random.default_rng(b).integers(
                0, self.new[b], rows)})
            t, (out, mean_abs, score_abs) = self.oracle(b, pick)
            lim = chunk.attention_bound(out, mean_abs, score_abs)
            err = np.abs(got[self.base[b] + t] - out)
            bad = ~(err <= lim)
            assert not bad.any(), (f"request {b} (seq {self.seq[b]}, new {self.new[b]}): {bad.sum()} of {bad.size} "
                                   f"outside the bound, largest error {np.nanmax(err):.3e}, "
                                   f"first at {np.argwhere(bad)[0]}")
