"""Float64 numpy oracle of the serving operators, from their definitions: rotation
at positions, the paged e4m3 cache, attention over it, causal attention of packed
prompts. Test infrastructure; shares no code with the CUDA library.

Each attention also returns the sums that error bounds are made of: per output the
sum of p |v|, and per row the largest sum of |q| |k| s over the keys it sees.
"""
from __future__ import annotations

import numpy as np

TOP = 448.0


def rope(x, positions, cos, sin, layout, transpose=False):
    """x [T, heads, d]; cos, sin [positions, rot/2]."""
    x = np.asarray(x, np.float64)
    half = cos.shape[1]
    c = np.asarray(cos, np.float64)[positions][:, None]
    s = np.asarray(sin, np.float64)[positions][:, None] * (-1.0 if transpose else 1.0)
    y = x.copy()
    if layout == "half":
        ia, ib = np.arange(half), np.arange(half) + half
    else:
        ia, ib = 2 * np.arange(half), 2 * np.arange(half) + 1
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def round_e4m3(x):
    """To the nearest e4m3 value, ties to even, saturating; NaN stays."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        e = np.floor(np.log2(np.where(x == 0, 1.0, np.abs(x))))
        step = np.exp2(np.maximum(np.where(np.isfinite(e), e, 0), -6) - 3)
        r = np.rint(x / step) * step
    r = np.where(np.isinf(x), np.sign(x) * TOP, r)
    return np.clip(r, -TOP, TOP)


def needed_exp(values):
    """Smallest e in [-32, 32] with |x| <= 448 2^e over the finite values."""
    v = np.abs(np.asarray(values, np.float64))
    v = v[np.isfinite(v)]
    top = v.max() if v.size else 0.0
    if top == 0.0:
        return -32
    e = int(np.ceil(np.log2(top / TOP)))
    while e > -60 and top <= TOP * 2.0 ** (e - 1):
        e -= 1
    while top > TOP * 2.0 ** e:
        e += 1
    return min(max(e, -32), 32)


def append(codes, scale, x, starts, cached, table):
    """Returns new (codes, scale) as float64 arrays: codes [pages, heads, page, d]
    values of the codes, scale [pages, heads]; x [T, heads, d]."""
    codes, scale = np.array(codes, np.float64), np.array(scale, np.float64)
    page = codes.shape[2]
    for b in range(len(cached)):
        n, a, e = int(cached[b]), int(starts[b]), int(starts[b + 1])
        t = a
        while t < e:
            p = n + t - a
            row, take = p % page, min(page - p % page, e - t)
            at = int(table[b][p // page])
            for h in range(codes.shape[1]):
                new = x[t:t + take, h]
                sc = 2.0 ** needed_exp(new)
                if row:
                    sc = max(sc, scale[at, h])
                    if sc != scale[at, h]:
                        codes[at, h, :row] = round_e4m3(codes[at, h, :row] * (scale[at, h] / sc))
                codes[at, h, row:row + take] = round_e4m3(new / sc)
                scale[at, h] = sc
            t += take
    return codes, scale


def softmax_rows(q, k, v, scale, seen):
    """q [n, d], k [m, d], v [m, d]; row i sees keys < seen[i]. Returns o, lse,
    sum p |v|, max over seen keys of scale sum |q| |k|, max p."""
    n, d = q.shape
    o, lse = np.zeros((n, d)), np.full(n, -np.inf)
    pv, qk, pm = np.zeros((n, d)), np.zeros(n), np.zeros(n)
    with np.errstate(all="ignore"):
        for i in range(n):
            m = int(min(max(seen[i], 0), k.shape[0]))
            if m == 0:
                continue
            x = scale * (k[:m] @ q[i])
            top = x.max()
            p = np.exp(x - top)
            total = p.sum()
            p /= total
            o[i] = p @ v[:m]
            lse[i] = top + np.log(total)
            pv[i] = p @ np.abs(v[:m])
            qk[i] = scale * (np.abs(k[:m]) @ np.abs(q[i])).max()
            pm[i] = p.max()
    return o, lse, pv, qk, pm


def cache_values(codes, scale, table_row, length):
    """The first `length` tokens of a sequence, [heads, length, d]."""
    page = codes.shape[2]
    pages = np.asarray(table_row)[: -(-length // page)] if length else np.zeros(0, int)
    x = np.asarray(codes, np.float64)[pages] * np.asarray(scale, np.float64)[pages][..., None, None]
    return x.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :length]


def cache_attn(q, k_codes, v_codes, k_scale, v_scale, lens, table, causal, scale):
    """q [B, n, H, d]. Returns o [B, n, H, d], lse [B, H, n], and the bounds' sums."""
    B, n, H, d = q.shape
    hkv = k_codes.shape[1]
    o, lse = np.zeros(q.shape), np.zeros((B, H, n))
    pv, qk, pm = np.zeros(q.shape), np.zeros((B, H, n)), np.zeros((B, H, n))
    for b in range(B):
        m = int(lens[b])
        k = cache_values(k_codes, k_scale, table[b], m)
        v = cache_values(v_codes, v_scale, table[b], m)
        seen = m - n + 1 + np.arange(n) if causal else np.full(n, m)
        for h in range(H):
            r = softmax_rows(np.asarray(q[b, :, h], np.float64), k[h // (H // hkv)], v[h // (H // hkv)], scale, seen)
            o[b, :, h], lse[b, h], pv[b, :, h], qk[b, h], pm[b, h] = r
    return o, lse, pv, qk, pm


def prompt_attn(q, k, v, starts, scale):
    """q [T, H, d], k, v [T, Hkv, d]. Returns o [T, H, d], lse [H, T], sums; rows
    outside the sequences are NaN."""
    T, H, d = q.shape
    o, lse = np.full((T, H, d), np.nan), np.full((H, T), np.nan)
    pv, qk, pm = np.zeros((T, H, d)), np.zeros((H, T)), np.zeros((H, T))
    group = H // k.shape[1]
    for a, e in zip(starts[:-1], starts[1:]):
        a, e = int(a), int(e)
        for h in range(H):
            r = softmax_rows(np.asarray(q[a:e, h], np.float64), np.asarray(k[a:e, h // group], np.float64),
                             np.asarray(v[a:e, h // group], np.float64), scale, 1 + np.arange(e - a))
            o[a:e, h], lse[h, a:e], pv[a:e, h], qk[h, a:e], pm[h, a:e] = r
    return o, lse, pv, qk, pm
