"""Long contexts that show a lost or doubled page.

The elementwise bound of a result grows with the mean of |v|, whatever the context, while results of normal
draws shrink with the root of its length.  Two checks whose signal does not shrink:

* planted keys: a row's own rotated query, at one slot of a chosen page, with a value far from the others'.
  Its length gives it about half of the row's weight, so that losing it moves the result by half of its value
  and counting it twice by a sixth;
* the error's norm over a (row, head) against the result's.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import chunk
from oracle.rope import rotate

PAGE = 16

# Values of normal draws have no preferred sign, so roundings add up by their squares.  A weight is rounded to
# bf16: at most 2^-8 of itself, uniform, a root mean square of 2^-8 / sqrt(3) at most; the result once more the
# same; the scores' fp16 operands (2^-11 / sqrt(3) of each rotated component) 2^-11 sqrt(2/3) |q k|, below
# 2^-10 for the rows' own keys: sqrt(2 (2^-8)^2 / 3 + 2^-20) = 0.0034 in all.  (Where one key has all the
# weight its rounding is no sum, but 2^-8 at most: sqrt(2^-16 + 2^-16 / 3 + 2^-20) = 0.0046.)  Over 64 or 128
# components a norm spreads by 9 % of its mean at most.  A page of 16 keys among n is sqrt(16 / n) of the norm
# of n like weights: 0.042 at 9000, 0.022 at 33,000.
NORM = 0.0065


def outside(got, out, mean_abs, score_abs):
    """None, or what of got [T][Hq][d] is outside the elementwise bound or the bound on norms."""
    err = np.abs(got - out)
    bad = ~(err <= chunk.attention_bound(out, mean_abs, score_abs))
    if bad.any():
        return f"{bad.sum()} of {bad.size} elements outside the bound, first {np.argwhere(bad)[0]}, by {np.nanmax(err):.3e}"
    size = np.linalg.norm(got - out, axis=-1) / np.maximum(np.linalg.norm(out, axis=-1), 1e-30)
    if not (size <= NORM).all():
        return f"error of {np.nanmax(size):.4f} of the norm at {np.unravel_index(np.nanargmax(size), size.shape)}"
    return None


def planted_key(q, q_pos, k_pos, n, theta):
    """The unrotated key at k_pos whose score with q (one head's query at q_pos) is ln n + |q|^2 / 2d, the
    logarithm of what n normal keys' exponentials add up to."""
    q = np.asarray(q, dtype=np.float64)
    d = q.shape[-1]
    size = (q @ q) / np.sqrt(d)
    score = np.log(n) + (q @ q) / (2 * d)
    return rotate(q[None, None], np.array([q_pos - k_pos]), theta)[0, 0] * (score / size)


def planted_value(d, i):
    v = np.full(d, 4.0)
    v[(np.arange(d) >> (i % 5)) & 1 == 1] = -4.0
    return v


def plant(c, b, pages, rows):
    """Into ChunkCase c, request b: a key for every (row, query head) of `rows`, the pages in turn (of those
    the row sees).  Slots differ within a kv head."""
    g = c.hq // c.hkv
    used = [set() for _ in range(c.hkv)]
    n_pages = -(-(c.seq[b] + c.new[b]) // PAGE)
    i = 0
    for t in rows:
        q_row = c.base[b] + t
        for h in range(c.hq):
            limit = c.seq[b] + t + 1                   # slots the row sees
            for _ in range(len(pages)):
                p = pages[i % len(pages)] % n_pages
                i += 1
                free = [j for j in range(p * PAGE, min((p + 1) * PAGE, limit)) if j not in used[h // g]]
                if free:
                    break
            else:
                continue
            j = free[(7 * i) % len(free)]
            used[h // g].add(j)
            pos = int(c.pp[b, j // PAGE]) + j % PAGE
            key = planted_key(c.q[q_row, h].double().numpy(), int(c.where[q_row]), pos, limit, c.theta)
            key, value = torch.from_numpy(key).to(torch.bfloat16), torch.from_numpy(planted_value(c.d, i)).to(torch.bfloat16)
            if j >= c.seq[b]:
                at = c.base[b] + j - c.seq[b]
                c.k_new[at, h // g], c.v_new[at, h // g] = key, value
            else:
                c.k_pool[c.bt[b, j // PAGE], h // g, j % PAGE] = key
                c.v_pool[c.bt[b, j // PAGE], h // g, j % PAGE] = value
