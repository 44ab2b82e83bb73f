"""Speculative decoding and cross attention over the cache, by definition (fp64, plain loops).

Test infrastructure only (see the package header).

* ``visible(n, length, parents)``: what draft i (position length - n + i) sees: every position before the
  drafts, its ancestors and itself; ``parents`` None is a chain.
* ``block_attention``: softmax attention of query blocks over a dequantized cache (OptR Eqs. 1-2, 5, 22, 27)
  under such a mask; rows that see nothing are zero.
* ``plan_pages`` / ``commit``: the page bookkeeping and the moves of accepted records, one item at a time.

Pinned by tests/test_oracle_tree.py: a chain equals causal_attention, a path of a tree equals decoding that
path alone, plans conserve pages, a commit equals writing the accepted tokens directly.
"""
from __future__ import annotations

import numpy as np

D = 128


def visible(n: int, length: int, parents=None) -> np.ndarray:
    """[n, length] truth values."""
    see = np.zeros((n, length), bool)
    base = length - n
    see[:, :base] = True
    for i in range(n):
        j = i
        while j >= 0:
            see[i, base + j] = True
            j = j - 1 if parents is None else int(parents[j])
    return see


def block_attention(q, k_hat, v_hat, r_k, gqa: int, see=None):
    """q [n, H_q, 128]; k_hat, v_hat [L, H_kv, 128] (rotated basis); see [n, L] or None (all).

    Returns o_rot [n, H_q, 128] and, for error bounds, the same sum over |v_hat| and max |logit| scale
    ||q'|| ||k_hat|| / sqrt(128) over the visible positions, [n, H_q]."""
    q = np.asarray(q, np.float64)
    n, hq, _ = q.shape
    length = k_hat.shape[0]
    see = np.ones((n, length), bool) if see is None else see
    out, mag, size = np.zeros((n, hq, D)), np.zeros((n, hq, D)), np.zeros((n, hq))
    for j in range(hq):
        h = j // gqa
        qr = q[:, j] @ r_k[h]
        for i in range(n):
            s = np.flatnonzero(see[i])
            if s.size == 0:
                continue
            k, v = k_hat[s, h], v_hat[s, h]
            a = k @ qr[i] / np.sqrt(D)
            p = np.exp(a - a.max())
            p /= p.sum()
            out[i, j] = p @ v
            mag[i, j] = p @ np.abs(v)
            size[i, j] = np.linalg.norm(qr[i]) * np.linalg.norm(k, axis=1).max() / np.sqrt(D)
    return out, mag, size


def plan_pages(page: int, num_blocks: int, old, new, table, ring, head: int, tail: int, max_new: int):
    """(table, ring, head, tail, cu_new, slots) after the plan; the arrays are copies."""
    table, ring = np.array(table), np.array(ring)
    held = lambda x: -(-int(x) // page)  # noqa: E731
    taken = sum(max(0, held(b) - held(a)) for a, b in zip(old, new))
    given = sum(max(0, held(a) - held(b)) for a, b in zip(old, new))
    tokens = sum(max(0, int(b) - int(a)) for a, b in zip(old, new))
    limit = table.shape[1] * page
    bad = any(not (0 <= x <= limit) for x in [*map(int, old), *map(int, new)])
    bad = bad or not (0 <= head <= tail <= head + num_blocks) or taken > tail - head
    bad = bad or tail - head + given > num_blocks or tokens > max_new
    slots = np.full(max_new, -1, np.int64)
    if bad:
        return table, ring, head, tail, np.zeros(len(old) + 1, np.int64), slots
    cu, back, at = [0], [], head
    for b, (o, n) in enumerate(zip(map(int, old), map(int, new))):
        for i in range(held(o), held(n)):
            table[b, i] = ring[at % num_blocks]
            at += 1
        back += [table[b, i] for i in range(held(n), held(o))]
        for pos in range(o, n):
            slots[cu[-1] + pos - o] = int(table[b, pos // page]) * page + pos % page
        cu.append(cu[-1] + max(0, n - o))
    for i, x in enumerate(back):
        ring[(tail + i) % num_blocks] = x
    return table, ring, at, tail + len(back), np.array(cu), slots


def commit(pool, n_kv_heads: int, page: int, cu, accepted, n_accepted, slots, lens):
    """(pool, new_lens): the accepted drafts' records moved to the first drafts' slots."""
    before = np.asarray(pool).reshape(-1, n_kv_heads, 72 * page)
    after = before.copy()
    new = []
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        for i in range(int(n_accepted[b])):
            src, dst = int(slots[cu[b] + accepted[b][i]]), int(slots[cu[b] + i])
            for base, width in ((0, 32), (32 * page, 32), (64 * page, 4), (68 * page, 4)):
                s, d = base + width * (src % page), base + width * (dst % page)
                after[dst // page, :, d:d + width] = before[src // page, :, s:s + width]
        new.append(int(lens[b]) - n + int(n_accepted[b]))
    return after.reshape(-1), np.array(new)
