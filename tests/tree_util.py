"""A batch of requests that draft trees on a page pool: seeded inputs, the calls, the oracle's answer."""
from __future__ import annotations

import numpy as np
import torch

import position_independent_kv_critical_gb300 as pcf
from oracle import chunk, tree

from chunk_util import PAGE, ChunkCase


def random_tree(n, rng, width=None, roots=False):
    """Parents of n nodes: each goes on from one of the `width` before it (None: any), or from the held
    tokens."""
    return [-1 if t == 0 or (roots and rng.random() < 0.2) else int(rng.integers(0 if width is None else max(0, t - width), t))
            for t in range(n)]


def chain(n):
    return list(range(-1, n - 1))


def star(n):
    return [-1] + [0] * (n - 1)


class TreeCase(ChunkCase):
    """ChunkCase whose request b brings the tree parents[b]."""

    def __init__(self, seq, parents, vocab=5, roots=False, **kw):
        self.parents = [list(p) for p in parents]
        super().__init__(seq, [len(p) for p in parents], **kw)
        rng = np.random.default_rng(kw.get("seed", 1) + 77)
        self.parent = np.array([p for t in self.parents for p in t] + [9] * (self.max_rows - self.rows), dtype=np.int32)
        self.draft = rng.integers(0, vocab, self.max_rows)
        self.choice = rng.integers(0, vocab, self.max_rows)
        self.root = rng.integers(0, vocab, self.n) if roots else None
        start = [int(self.where[a]) if e > a else 0 for a, e in zip(self.base[:-1], self.base[1:])]
        self.words = (self.max_chunk + 31) // 32
        self.node_pos, self.bits = tree.tables(self.parents, start, self.words)

    def to_device(self):
        super().to_device()
        i32 = lambda x: None if x is None else torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()
        self.tree = pcf.DraftTree(self.L)
        self.d_parent, self.d_draft, self.d_choice, self.d_root = (i32(x) for x in (self.parent, self.draft, self.choice,
                                                                                   self.root))
        self.ws = torch.empty(max(16, self.tree.attention_workspace_bytes()), dtype=torch.uint8, device="cuda")
        return self

    def tables(self, **kw):
        super().tables(**kw)
        pcf.tree_tables(self.L, self.tree, self.d_parent, **kw)

    def append(self, **kw):
        pcf.append_kv(self.L, self.dkn, self.dvn, self.dk, self.dv, **kw)

    def attend(self, **kw):
        pcf.tree_attention(self.L, self.tree, self.dq, self.dk, self.dv, self.rope, self.out, self.ws, excl=self.d_excl,
                           **kw)

    def accept(self, **kw):
        pcf.tree_accept(self.L, self.tree, self.d_parent, self.d_draft, self.d_choice, self.d_free, self.d_seq_out,
                        self.d_head_out, root_choice=self.d_root, **kw)

    # ---- oracle side
    def oracle(self, b, rows=None):
        s, n = self.seq[b], self.seq[b] + self.new[b]
        k, v = self.k_pool.double().numpy().copy(), self.v_pool.double().numpy().copy()
        sl = slice(self.base[b], self.base[b + 1])
        page, r = self.slots[sl] // PAGE, self.slots[sl] % PAGE
        k[page, :, r] = self.k_new[sl].double().numpy()
        v[page, :, r] = self.v_new[sl].double().numpy()
        pages = self.bt[b, : -(-n // PAGE)]
        pos = (self.pp[b, : len(pages), None] + np.arange(PAGE)).reshape(-1)[:n].astype(np.int64)
        pos[s:] = self.node_pos[sl]
        K, V = chunk.gather(k, pages, n), chunk.gather(v, pages, n)
        seen = np.zeros((self.new[b], n), dtype=bool)
        seen[:, :s] = True
        for t, line in enumerate(tree.lines(self.parents[b])):
            seen[t, [s + u for u in line]] = True
        if self.excl is not None:
            gone = ((self.excl[b, : len(pages), None].astype(np.int64) >> np.arange(PAGE)) & 1).reshape(-1)[:n]
            seen = seen & (gone == 0)[None]
        K = np.where(seen.any(axis=0)[:, None, None], K, 0.0)
        t = np.arange(self.new[b]) if rows is None else np.asarray(rows)
        q = self.q[sl].double().numpy()[t]
        return t, chunk.attention(q, self.node_pos[sl][t], K, V, pos, seen[t], self.theta)

    def accepted(self):
        return tree.accept(self.seq, self.parents, self.draft, self.choice, self.root, self.bt, self.free, 0, self.head)
