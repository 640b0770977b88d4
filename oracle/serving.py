"""Plain restatement of the serving operators (numpy, 64 bits; test infrastructure only).

rotate_rows      the rotary position of keys and queries, in fp64 or, step by
                 step as the operator defines it, in fp32
paged_attention  attention of one new token per request over a paged cache
lora             low-rank adapters of many requests beside a projection
"""

from __future__ import annotations

import numpy as np


def rotate_rows(x, cos, sin, rot, interleaved, dtype=np.float64):
    """x [T, heads, dim]; cos, sin [T, rot / 2]. Every product and sum is one operation of `dtype`."""
    x = np.array(x, dtype=dtype)
    if rot == 0:
        return x
    c = np.asarray(cos, dtype=dtype)[:, None, :]
    s = np.asarray(sin, dtype=dtype)[:, None, :]
    if interleaved:
        i = slice(0, rot, 2)
        j = slice(1, rot, 2)
    else:
        i = slice(0, rot // 2)
        j = slice(rot // 2, rot)
    a, b = x[..., i].copy(), x[..., j].copy()
    x[..., i] = a * c - b * s
    x[..., j] = b * c + a * s
    return x


def gather(cache, table, n, begin=0):
    """cache [pages, heads, page_size, dim], table [max_pages] -> the tokens begin .. n - 1 as [heads, n - begin, dim]."""
    page = cache.shape[2]
    return np.stack([cache[table[j // page], :, j % page] for j in range(begin, n)], axis=1) if n > begin else \
        np.zeros((cache.shape[1], 0, cache.shape[3]))


def paged_attention(q, k, v, table, lens, scale, window=0):
    """q [B, q_heads, dim]; k, v [pages, kv_heads, page_size, dim] -> (out, lse, bound) in fp64.

    bound[b, h] carries what the rounding bound of an fp32 evaluation needs:
    (max_j scale sum_i |q_i k_ji|, sum_j p_j |v_j| / sum_j p_j per channel).
    """
    B, hq, d = q.shape
    group = hq // k.shape[1]
    out = np.zeros((B, hq, d))
    lse = np.full((B, hq), -np.inf)
    top = np.zeros((B, hq))
    absv = np.zeros((B, hq, d))
    for b in range(B):
        n = int(lens[b])
        begin = max(0, n - window) if window else 0
        if n == begin:
            continue
        kb, vb = gather(k, table[b], n, begin), gather(v, table[b], n, begin)
        for h in range(hq):
            kh, vh = kb[h // group], vb[h // group]
            s = scale * (kh @ q[b, h])
            m = s.max()
            p = np.exp(s - m)
            out[b, h] = p @ vh / p.sum()
            lse[b, h] = m + np.log(p.sum())
            top[b, h] = abs(scale) * (np.abs(kh) @ np.abs(q[b, h])).max()
            absv[b, h] = p @ np.abs(vh) / p.sum()
    return out, lse, (top, absv)


def lora(x, base, A, B, scale, ids):
    """base[m] + scale[a] B[a] (A[a] x[m]) with a = ids[m]; rows with ids[m] < 0 are base's. Returns (y, bound):
    bound[m, n] = scale sum_r |B[a]| (|A[a]| |x[m]|), the magnitude that rounding errors are relative to."""
    y = np.array(base, dtype=np.float64)
    bound = np.zeros_like(y)
    for m, a in enumerate(ids):
        if a >= 0:
            y[m] += scale[a] * (B[a] @ (A[a] @ x[m]))
            bound[m] = abs(scale[a]) * (np.abs(B[a]) @ (np.abs(A[a]) @ np.abs(x[m])))
    return y, bound
