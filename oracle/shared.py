"""Plain fp64 numpy form of skv_shared_attend, written from the formulas in
include/sparsekv.h; used by the tests only."""
from __future__ import annotations

import numpy as np


def shared_attend(q, k, v, group_start, prefix_table, prefix_lengths, block_table, page, lengths, scale, starts):
    """q fp64 [n][Hq][d]; k, v fp64 [rows][Hkv][d]; starts: B + 1 token offsets.  Returns (out, spread): the output and
    sum_t w_t |v_t|, fp64 [n][Hq][d]; tokens of no request are NaN.  Pages < 0 or past the pool are left out."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out, spread = np.full((2, n, Hq, d), np.nan)

    def rows(pages, T):
        t = np.arange(min(max(int(T), 0), len(pages) * page))
        blk = np.asarray(pages)[t // page].astype(np.int64) if len(t) else t
        there = (blk >= 0) & (blk < len(k) // page)
        return (blk * page + t % page)[there], t[there]

    for b, T in enumerate(lengths):
        lo, hi = int(starts[b]), int(starts[b + 1])
        pre = np.zeros(0, np.int64)
        for g, P in enumerate(prefix_lengths):
            if group_start[g] <= b < group_start[g + 1]:
                pre, _ = rows(prefix_table[g], P)
        own, t = rows(block_table[b], T)
        for i in range(lo, hi):
            at = np.concatenate([pre, own[t <= int(T) - (hi - lo) + i - lo]])
            for h in range(Hkv):
                hq = slice(h * G, h * G + G)
                vv = v[at, h]
                with np.errstate(invalid="ignore"):
                    z = q[i, hq] @ k[at, h].T * scale
                    top = z.max(1, keepdims=True, initial=-np.inf)
                    w = np.exp(z - np.where(np.isfinite(top), top, 0.0))
                    tot = w.sum(1, keepdims=True)
                    w = w / np.where(tot > 0, tot, 1.0)
                    out[i, hq], spread[i, hq] = w @ vv, w @ np.abs(vv)
    return out, spread
