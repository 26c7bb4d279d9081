"""Trees of drafted tokens on the position-free pool, in fp64 and node by node (oracle; test
infrastructure only).

Source: MiniPIC, section 2.1 (keys stay unrotated, a request brings the positions).  The pages draft
nothing: the reading is the common one, a node's position follows from its depth, it sees the held
tokens, itself and the nodes it goes on from, and the branch whose tokens the model itself chooses is
kept.
"""
from __future__ import annotations

import numpy as np

PAGE = 16


def lines(parent):
    """For every node the nodes it goes on from, in order, itself last."""
    out = []
    for t, p in enumerate(parent):
        out.append((out[p] if p >= 0 else []) + [t])
    return out


def tables(parents, start, words):
    """Positions [rows] and bits [rows][words] (uint32) of all requests' trees, request after request."""
    pos, bits = [], []
    for parent, first in zip(parents, start):
        for line in lines(parent):
            pos.append(int(first) + len(line) - 1)
            word = [0] * words
            for u in line:
                word[u // 32] |= 1 << (u % 32)
            bits.append(word)
    return np.array(pos, dtype=np.int64), np.array(bits, dtype=np.uint32).reshape(-1, words)


def branch(parent, draft, choice, root=None):
    """The nodes that are kept, in order, and the token chosen behind the last one (-1: none known)."""
    at, said, kept = -1, root, []
    while True:
        on = [t for t, p in enumerate(parent) if p == at and (draft[t] == said if kept or root is not None else t == 0)]
        if not on:
            return kept, -1 if said is None else int(said)
        at = on[0]
        said = choice[at]
        kept.append(at)


def accept(seq, parents, draft, choice, root, block_table, free, head, taken):
    """(path, n_kept, next_token, seq_out, free, head) of a batch whose chunk took `taken` pages from
    free[head:]."""
    path, kept, token, length, back, used, base = [], [], [], [], [], 0, 0
    free = list(free)
    for b, parent in enumerate(parents):
        n = len(parent)
        mine, said = branch(parent, draft[base: base + n], choice[base: base + n], None if root is None else root[b])
        path += mine + [-1] * (n - len(mine))
        kept.append(len(mine))
        token.append(said)
        s = int(seq[b])
        length.append(s + len(mine))
        held, enough, had = (-(-x // PAGE) for x in (s, s + len(mine), s + n))
        used += enough - held
        back += [int(x) for x in block_table[b][enough: had]]
        base += n
    assert used + len(back) == taken
    free[head + used: head + taken] = back
    return path, kept, token, length, free, head + used


def keep(pool, seq, row_base, path, kept, block_table):
    """The pool [pages][Hkv][16][...] with every branch's entries behind the held ones."""
    pool = np.array(pool)
    before = pool.copy()
    for b in range(len(seq)):
        for i in range(kept[b]):
            a, z = int(seq[b]) + path[row_base[b] + i], int(seq[b]) + i
            pool[block_table[b][z // PAGE], :, z % PAGE] = before[block_table[b][a // PAGE], :, a % PAGE]
    return pool
