"""Continuing a request on the position-free pool, in fp64 and token by token (oracle; test
infrastructure only).

Source: MiniPIC, section 2.1 (keys stay unrotated in shared pages, every request brings its own
logical positions) and QCFuse, Phase 4 (the request goes on from the merged cache).  The pages give
no tables: the reading is the common one, sixteen slots to a page, new pages from a list of free
ones in request order.
"""
from __future__ import annotations

import numpy as np

from .rope import rotate

PAGE = 16


def tables(seq, new, free, head, block_table, page_pos, next_pos=None):
    """Grow request b from seq[b] by new[b] tokens.  Returns (block_table, page_pos, slots, positions,
    row_base, head): copies of the tables with the started pages, one slot (page * 16 + r) and one
    position for every row, the first row of every request, the list's new head."""
    bt, pp = np.array(block_table), np.array(page_pos)
    slots, where, base = [], [], [0]
    for b in range(len(seq)):
        s = int(seq[b])
        if next_pos is not None:
            p = int(next_pos[b])
        elif s == 0:
            p = 0
        else:
            p = int(pp[b, (s - 1) // PAGE]) + (s - 1) % PAGE + 1
        for _ in range(int(new[b])):
            if s % PAGE == 0:
                bt[b, s // PAGE], pp[b, s // PAGE] = free[head], p
                head += 1
            slots.append(int(bt[b, s // PAGE]) * PAGE + s % PAGE)
            where.append(p)
            s, p = s + 1, p + 1
        base.append(len(slots))
    return bt, pp, np.array(slots, dtype=np.int64), np.array(where, dtype=np.int64), np.array(base), head


def appended(k, slot_pos, row_pos, theta):
    """The keys as they are stored, [rows][Hkv][d]: turned by row_pos - slot_pos."""
    return rotate(k, np.asarray(row_pos) - np.asarray(slot_pos), theta)


def gather(pool, pages, n):
    """The first n tokens of a request's pages: [n][Hkv][d]."""
    return np.asarray(pool, dtype=np.float64)[pages].transpose(0, 2, 1, 3).reshape(-1, pool.shape[1], pool.shape[3])[:n]


def attention(q, q_pos, k, v, k_pos, seen, theta):
    """out [T][Hq][d] of rows q [T][Hq][d] at q_pos over keys k, values v [n][Hkv][d] at k_pos, row t
    taking part with the keys where seen[t]; and for a bound on errors, per (row, head), the weighted
    mean of |v| and of sum_i |q_i k_i| / sqrt(d) taken at its largest key."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    T, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    qr, kr = rotate(q, q_pos, theta), rotate(k, k_pos, theta)
    out, mean_abs, score_abs = np.zeros((T, hq, d)), np.zeros((T, hq, d)), np.zeros((T, hq))
    for h in range(hq):
        kh, vh = kr[:, h // g], v[:, h // g]
        s = np.where(seen, qr[:, h] @ kh.T / np.sqrt(d), -np.inf)
        big = np.where(seen, np.abs(qr[:, h]) @ np.abs(kh).T / np.sqrt(d), 0.0)
        top = s.max(axis=1, keepdims=True)
        w = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        total = w.sum(axis=1, keepdims=True)
        w = w / np.where(total == 0, 1.0, total)
        vh = np.where(seen.any(axis=0)[:, None], vh, 0.0)     # what no row sees may be anything
        out[:, h], mean_abs[:, h] = w @ vh, w @ np.abs(vh)
        score_abs[:, h] = big.max(axis=1)
    return out, mean_abs, score_abs


def attention_bound(out, mean_abs, score_abs, bf16_weights=True):
    """Largest error of a result rounded to bf16 whose products take fp16 rotated operands and whose
    weights are rounded to bf16 before they meet the values.

    A rotated query and key are each within 2^-11 relative of their values (fp16, half a step), a
    score then within e = 2 * 2^-11 * sum|q_i k_i| / sqrt(d) (the cross term below 2^-22 of it) plus
    2^-20 of the same sum for fp32 products, sums and angles; a weight within exp(2 e) - 1 <= 2.1 e
    of itself after normalisation (numerator and denominator), and within 2^-8 (half a step of bf16)
    of that where it is rounded, so the weighted sum is off by at most (2.1 e + 2 * 2^-8) sum w|v|
    (rounded weights over a sum of unrounded ones or of rounded ones alike); the result is rounded
    once more, 2^-8 of itself.  2^-14 sum w|v| covers the fp32 sums, exponentials (2 units in the
    last place) and partial results of a split row."""
    e = (2.0 ** -10 + 2.0 ** -20) * score_abs[..., None]
    rel = 2.1 * e + (2 * 2.0 ** -8 if bf16_weights else 0.0) + 2.0 ** -14
    return (1 + 2.0 ** -8) * rel * mean_abs + 2.0 ** -8 * np.abs(out) + 1e-30
