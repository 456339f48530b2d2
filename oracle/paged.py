"""fp64 oracle of the paged K/V cache operators (test infrastructure only).

Definitions (numpy, loops over requests and heads):

* plan: request r holds ``cached[r]`` tokens on ceil(cached / ps) pages and needs
  ceil((cached + new) / ps); the missing ones come from the front of the free list,
  requests in order.
* attend: the n new tokens of request r are the last n of its kv tokens; the one at
  position i sees key j iff 0 <= j <= i, j < kv, j > i - W under a window of W keys, and,
  with selected blocks, j // bs is one of the row's block numbers.
"""
from __future__ import annotations

import numpy as np


def plan(new, cached, free, table, ps, total):
    """(cu, kv_lens, slots, positions, used, table) of one step; -1 for missing pages."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    free = [int(x) for x in free]
    cu, kv, slots, positions, used = [0], [], [], [], 0
    for r, (a, b) in enumerate(zip(new, cached)):
        a, b = max(int(a), 0), max(int(b), 0)
        for c in range(min(-(-b // ps), width), min(-(-(a + b) // ps), width)):
            table[r, c] = free[used] if used < len(free) else -1
            used += 1
        cu.append(cu[-1] + a)
        kv.append(a + b)
        for p in range(b, b + a):
            page = table[r, p // ps] if p // ps < width else -1
            slots.append(-1 if page < 0 else page * ps + p % ps)
            positions.append(p)
    slots, positions = slots[:total], positions[:total]
    pad = total - len(slots)
    return (np.array(cu, np.int32), np.array(kv, np.int32), np.array(slots + [-1] * pad, np.int64),
            np.array(positions + [0] * pad, np.int32), used, table.astype(np.int32))


def gather(cache, table_row, n, ps):
    """Rows 0 .. n - 1 of one request out of a [pages, ps, hkv, d] cache."""
    j = np.arange(n)
    return cache[table_row[j // ps], j % ps]


def attend(q, k_cache, v_cache, cu, kv_lens, table, scale, window=0, block_idx=None, block_size=0):
    """(out [T, hq, d], lse [hq, T], bound [T, hq, d]); bound = softmax weights times |V|,
    what an error in the weights is measured against.  Rows outside the requests: 0, -inf."""
    T, hq, d = q.shape
    hkv, ps = k_cache.shape[2], k_cache.shape[1]
    G = hq // hkv
    out, bound = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse = np.full((hq, T), -np.inf)
    for r, kv in enumerate(kv_lens):
        a, b, kv = int(cu[r]), int(cu[r + 1]), int(kv)
        if a == b:
            continue
        K = gather(k_cache, table[r], kv, ps).astype(np.float64)
        V = gather(v_cache, table[r], kv, ps).astype(np.float64)
        i = kv - (b - a) + np.arange(b - a)
        j = np.arange(kv)
        seen = j[None, :] <= i[:, None]
        if window > 0:
            seen &= j[None, :] > i[:, None] - window
        V = np.where(seen.any(0)[:, None, None], V, 0.0)   # rows nobody sees may hold anything
        for g in range(hkv):
            mine = seen
            if block_idx is not None:
                mine = np.zeros_like(seen)
                for t in range(b - a):
                    for blk in block_idx[a + t, g]:
                        if 0 <= blk <= i[t] // block_size:
                            mine[t, blk * block_size:(blk + 1) * block_size] = True
                mine &= seen
            vis = mine.any(0)
            Vg = np.where(vis[:, None], V[:, g], 0.0)
            for h in range(g * G, (g + 1) * G):
                s = np.where(mine, scale * (q[a:b, h].astype(np.float64) @ np.where(vis[:, None], K[:, g], 0.0).T),
                             -np.inf)
                m = s.max(1, initial=-np.inf)
                p = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None])
                total = p.sum(1)
                w = p / np.where(total > 0, total, 1.0)[:, None]
                out[a:b, h] = w @ Vg
                bound[a:b, h] = w @ np.abs(Vg)
                with np.errstate(divide="ignore"):
                    lse[h, a:b] = np.where(total > 0, np.where(np.isfinite(m), m, 0.0) + np.log(total), -np.inf)
    return out, lse, bound
