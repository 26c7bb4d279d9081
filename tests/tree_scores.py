"""Requests whose scores grow along the context, so that a row's reference moves behind its first unit.

The attention of a tree keeps a row's softmax reference from the first scores it sees and moves it when 32 weights
add up to more than 2^16 times that of the first scores' largest (rounded up to a power of two); what the row has summed up by then is scaled down by a power of two.  Normal
draws never get there.  Here two dimensions that hardly turn (the two lowest frequencies) carry a chosen level, in
bits, from a slot to the rows of three kinds: kind 0 sees level a, kind 1 level b, kind 2 the sum of both.  A node's
query heads go through the kinds in turn, so the rows of one warp move at different places.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import tree
from oracle.rope import rotate

from chunk_util import PAGE
from tree_util import TreeCase, random_tree

UNIT, HALF = 64, 32
SIZE = 4.0           # of a row's query in its dimension
NOISE = 0.3          # of everything else in queries and keys
MOVE = 65536.0       # sum of 32 weights that moves a reference


def leveled(levels, nodes, hq=8, hkv=2, d=64, seed=1, excl=None):
    """One request a list of levels: {slot: (a, b)}, over `slots` held tokens (its key "slots")."""
    rng = np.random.default_rng(seed)
    c = TreeCase([v["slots"] for v in levels], [random_tree(n, rng, 9) for n in nodes], hq=hq, hkv=hkv, d=d, seed=seed,
                 stale="normal")
    ia, ib = d // 2 - 1, d // 2 - 2
    bits = np.log(2.0) * np.sqrt(d) / SIZE             # of a key's dimension, for a level of one bit
    for t in (c.q, c.k_pool, c.k_new):
        t.mul_(NOISE)
        t[..., ia] = t[..., ib] = t[..., ia + d // 2] = t[..., ib + d // 2] = 0.0
    kind = kinds(c)
    c.q[..., ia] = torch.from_numpy(np.where(kind != 1, SIZE, 0.0)).to(torch.bfloat16)
    c.q[..., ib] = torch.from_numpy(np.where(kind != 0, SIZE, 0.0)).to(torch.bfloat16)
    for b, v in enumerate(levels):
        for j, (a, z) in v["at"].items():
            page, r = c.bt[b, j // PAGE], j % PAGE
            c.k_pool[page, :, r, ia], c.k_pool[page, :, r, ib] = a * bits, z * bits
            # (a value of its own sign for every slot that has a level: 3 or -3, by the dimension)
            flip = np.where((np.arange(d) >> (j % 5)) & 1 == 1, -3.0, 3.0)
            c.v_pool[page, :, r] = torch.from_numpy(flip).to(torch.bfloat16)
    return c


def kinds(c):
    return (np.arange(c.max_rows)[:, None] + np.arange(c.hq)[None]) % 3


def pair(j, level):
    """A slot for kind 0 and the one behind it for kind 1, each of that level (kind 2 sees both)."""
    return {j: (level, 0.0), j + 1: (0.0, level)}


def moves_once(unit, half, second=None):
    """Levels of a request of seven units: weights of 2^14.9 in the second halves of units 0 and 1, then keys of
    level 18 in one half of `unit`; for `second` (a unit, a half) keys of 18 more behind it, with weights of a
    quarter of theirs between."""
    at = {**pair(40, 14.9), **pair(UNIT + 41, 14.9), **pair(UNIT * unit + HALF * half + 7, 18.0)}
    if second is not None:
        u, h = second
        at.update(pair(UNIT * u + HALF * h + 19, 36.0))
        for w in range(unit + 1, u):
            at.update(pair(UNIT * w + 50, 32.0))
    return dict(slots=7 * UNIT - 25, at=at)


def both_halves(unit):
    """Kind 0 moves in the first half of `unit`, kind 1 in the second (kind 2 in the first too)."""
    return dict(slots=7 * UNIT - 25, at={**pair(40, 14.9), **pair(UNIT + 41, 14.9), UNIT * unit + 5: (18.0, 0.0),
                                         UNIT * unit + HALF + 9: (0.0, 18.0)})


# ------------------------------------------------------------------ the loop over units, on the CPU
def scores(c, b, rows):
    """Scores [rows][Hq][n] in bits of request b, -inf where hidden, and its values [n][Hkv][d]."""
    s, n = c.seq[b], c.seq[b] + c.new[b]
    sl = slice(c.base[b], c.base[b + 1])
    pages = c.bt[b, : -(-n // PAGE)]
    flat = lambda pool, new: np.concatenate([
        pool[pages].double().numpy().transpose(0, 2, 1, 3).reshape(-1, c.hkv, c.d)[:s], new[sl].double().numpy()])
    K, V = flat(c.k_pool, c.k_new), flat(c.v_pool, c.v_new)
    pos = (c.pp[b, : len(pages), None] + np.arange(PAGE)).reshape(-1)[:n].astype(np.int64)
    pos[s:] = c.node_pos[sl]
    kr = rotate(K, pos, c.theta)
    qr = rotate(c.q[sl].double().numpy()[rows], c.node_pos[sl][rows], c.theta)
    g = c.hq // c.hkv
    x = np.einsum("thd,nhd->thn", qr, np.repeat(kr, g, axis=1)) / np.sqrt(c.d) / np.log(2.0)
    lines = tree.lines(c.parents[b])
    for i, t in enumerate(rows):
        x[i, :, [s + u for u in range(c.new[b]) if u not in lines[t]]] = -np.inf
    return x, V


def run(x, v, units, mistake=None):
    """One row: its sum over `units` in order, kept against a reference that moves as the kernel's does, and where
    it moved behind the first unit: (unit, half, factor).  `mistake`: "kept" leaves the result as it was when the
    reference moves, "first" only when it moves again in the same unit's second half, "half" leaves the weights of
    the first half."""
    ref, total, out, moved = -np.inf, 0.0, np.zeros(v.shape[-1]), []
    for q, u in enumerate(units):
        held = np.zeros_like(out)                      # the first half's products, which come behind the second's scores
        for h in range(2):
            a = slice(UNIT * u + HALF * h, min(len(x), UNIT * u + HALF * (h + 1)))
            y = x[a]
            if y.size == 0:
                continue
            w = np.exp2(np.minimum(y - (ref if np.isfinite(ref) else 0.0), 1000.0))
            if (not np.isfinite(ref) or w.sum() > MOVE) and np.isfinite(y.max()):
                to = np.ceil(y.max())
                alpha = np.exp2(ref - to)
                if q > 0 and np.isfinite(ref):
                    moved.append((u, h, alpha))
                again = h == 1 and moved[-1:] and len(moved) > 1 and moved[-2][:2] == (u, 0)
                total *= alpha
                if mistake != "kept" and not (mistake == "first" and again):
                    out *= alpha
                if mistake != "half":
                    held *= alpha
                ref = to
                w = np.exp2(y - ref)
            total += w.sum()
            held += w @ v[a]
        out += held
    return ref, total, out, moved
