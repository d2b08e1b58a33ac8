"""Plain fp64 numpy forms of skv_norm_rope_append and skv_paged_attend, written
from the formulas in include/sparsekv.h; used by the tests only."""
from __future__ import annotations

import numpy as np


def norm_rope(x, weight, eps, positions, inv_freq, interleaved):
    """x fp64 [n][H][d] -> (z, mag): the normed, rotated heads, and for each value |y_a| + |y_b| of its pair
    (|y| outside the rotated dims), the scale of its rounding errors."""
    x = np.asarray(x, np.float64)
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    f = np.asarray(inv_freq, np.float64)
    rot = 2 * len(f)
    t = np.asarray(positions, np.float64)[:, None] * f[None, :]
    c, s = np.cos(t)[:, None, :], np.sin(t)[:, None, :]
    z, mag = y.copy(), np.abs(y)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return z, mag


def paged_attend(q, k, v, block_table, page, lengths, scale, starts, S, W):
    """q fp64 [n][Hq][d]; k, v fp64 [rows][Hkv][d]; starts: B + 1 token offsets.  Returns (out, spread): the output
    and sum_t w_t |v_t|, fp64 [n][Hq][d]; tokens behind the last request are NaN."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = np.full((n, Hq, d), np.nan)
    spread = np.full((n, Hq, d), np.nan)
    for b, T in enumerate(lengths):
        lo, hi = int(starts[b]), int(starts[b + 1])
        if hi == lo:
            continue
        T = int(T)
        t = np.arange(max(T, 0))
        p = T - (hi - lo) + np.arange(hi - lo)
        see = t[None, :] <= p[:, None]
        if W > 0:
            see &= (t[None, :] > p[:, None] - W) | (t[None, :] < S)
        used = see.any(0)
        t, see = t[used], see[:, used]
        rows = block_table[b][t // page].astype(np.int64) * page + t % page
        for g in range(Hq):
            kk, vv = k[rows, g // G], v[rows, g // G]
            with np.errstate(invalid="ignore"):
                z = np.where(see, q[lo:hi, g] @ kk.T * scale, -np.inf)
                top = z.max(1, keepdims=True, initial=-np.inf)
                w = np.where(see, np.exp(z - np.where(np.isfinite(top), top, 0.0)), 0.0)
            tot = w.sum(1, keepdims=True)
            w = w / np.where(tot > 0, tot, 1.0)
            if np.isfinite(vv).all():
                out[lo:hi, g] = w @ vv
                spread[lo:hi, g] = w @ np.abs(vv)
            else:  # a value that a token does not see takes no part, whatever it holds
                for i in range(hi - lo):
                    m = see[i]
                    with np.errstate(invalid="ignore"):
                        out[lo + i, g] = (w[i, m, None] * vv[m]).sum(0)
                        spread[lo + i, g] = (w[i, m, None] * np.abs(vv[m])).sum(0)
    return out, spread
