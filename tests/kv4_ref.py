"""The attention-layer operators over the paged 4-bit cache, plainly in NumPy fp64 from their definitions (include/gdn.h)."""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([e * 2.0 ** -9 if e < 8 else (8 + e % 8) * 2.0 ** (e // 8 - 10) for e in range(127)])


def nearest(x, grid):
    """Index of the grid value nearest to each x >= 0; ties to the even index, values beyond the end to the last."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def quantise(x, unit=1.0):
    """(codes uint8 [.., D/2], scales uint8 [.., D/16]) of x [.., D]; NaN counts as 0, infinities as the largest."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, np.clip(x, -1e300, 1e300))
    g = x.reshape(*x.shape[:-1], -1, 16)
    sb = nearest(np.abs(g).max(-1) / 6.0 / unit, E4M3)
    s = (E4M3[sb] * unit)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        mag = np.where(s > 0, nearest(np.where(s > 0, np.abs(g) / s, 0.0), E2M1), 0)
    code = (mag + 8 * (g < 0)).astype(np.uint8).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), sb.astype(np.uint8)


def numbers(codes, scales, unit=1.0):
    """The values of codes [.., D/2] and scales [.., D/16]."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    return v * np.repeat(E4M3[np.minimum(scales, 126)], 16, -1) * unit


def norm_rope(x, w, positions, inv_freq, eps, interleaved):
    """x [N, H, D] fp64 -> (y, s): the result, and |y_a| + |y_b| before the rotation (what its rounding scales with)."""
    D, H = x.shape[-1], len(inv_freq)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    a, b = (np.arange(0, 2 * H, 2), np.arange(1, 2 * H, 2)) if interleaved else (np.arange(H), H + np.arange(H))
    t = positions.astype(np.float64)[:, None, None] * inv_freq.astype(np.float64)
    out, size = y.copy(), np.abs(y)
    out[..., a] = y[..., a] * np.cos(t) - y[..., b] * np.sin(t)
    out[..., b] = y[..., b] * np.cos(t) + y[..., a] * np.sin(t)
    both = np.abs(y[..., a]) + np.abs(y[..., b])
    size[..., a] = both
    size[..., b] = both
    return out, size


def attention(q, k, v, limits, scale):
    """q [n, D], k, v [L, D], limits [n]: the keys each query sees -> (o, lse, bound of o's error, bound of lse's).

    The bounds count what the kernel's arithmetic may lose before o's own rounding: the scores' fp32 sums (D terms of
    2^-24 each, queries held to 2^-25 of their row's largest), the rounding of p to f16 (2^-11 of it, 2^-25 at least), and
    a few fp32 roundings of exponentials and sums."""
    n, D = q.shape
    o, lse = np.zeros((n, D)), np.full(n, -math.inf)
    be, bl = np.zeros((n, D)), np.zeros(n)
    for i in range(n):
        L = int(max(0, min(limits[i], len(k))))
        if L == 0:
            continue
        s = k[:L] @ q[i] * scale
        ds = abs(scale) * ((np.abs(k[:L]) @ np.abs(q[i])) * D * 2.0 ** -23
                           + np.abs(k[:L]).sum(-1) * np.abs(q[i]).max() * 2.0 ** -24) + np.abs(s) * 2.0 ** -21
        m = s.max()
        p = np.exp(s - m)
        l = p.sum()
        o[i] = p @ v[:L] / l
        lse[i] = m + math.log(l)
        rel = 2 * ds + 2.0 ** -20 + 2.0 ** -11
        be[i] = (p * rel) @ np.abs(v[:L]) / l + np.abs(o[i]) * float((p * (2 * ds + 2.0 ** -20)).sum() / l) \
            + L * 2.0 ** -25 * np.abs(v[:L]).max(0) / l
        bl[i] = float((p * (ds + 2.0 ** -20)).sum() / l) + 2.0 ** -22 * max(1.0, abs(lse[i]), abs(m)) + L * 2.0 ** -24
    return o, lse, be, bl


def page_plan(kv, new, page, tables, held, free, taken, N):
    """Everything gdn_page_plan writes, lane by lane."""
    B, width = tables.shape
    tables, held = tables.copy(), held.copy()
    cu, total = np.zeros(B + 1, np.int64), kv.copy()
    pos, slots = np.zeros(N, np.int32), np.full(N, -1, np.int32)
    upto, after, bits = 0, taken, 0
    ok_list = 0 <= taken <= len(free)
    left = len(free) - taken if ok_list else 0
    base = taken if ok_list else 0
    if not ok_list:
        bits |= 1
    for b in range(B):
        k, n, h = int(kv[b]), int(new[b]), int(held[b])
        cu[b + 1] = cu[b] + max(n, 0)
        fine = k >= 0 and n >= 0 and 0 <= h <= width and k + n <= width * page and h * page >= k
        got = False
        if fine:
            need = max(0, -(-(k + n) // page) - h)
            upto += need
            got = need == 0 or upto <= left
            if got:
                tables[b, h:h + need] = free[base + upto - need:base + upto]
                held[b] = h + need
                total[b] = k + n
                if need:
                    after = taken + upto
            else:
                bits |= 16
        else:
            bits |= 8
        for i in range(max(n, 0)):
            t = cu[b] + i
            if t >= N:
                break
            pos[t] = k + i
            if got:
                pg = tables[b, (k + i) // page]
                if 0 <= pg < len(free):
                    slots[t] = pg * page + (k + i) % page
                else:
                    bits |= 1
    if cu[B] > N:
        bits |= 8
    return tables, cu.astype(np.int32), pos, slots, total, held, np.int32(after), bits
