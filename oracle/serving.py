"""Plain restatement of the serving operators (numpy, 64 bits; test infrastructure only).

rotate_rows      the rotary position of keys and queries, in fp64 or, step by
                 step as the operator defines it, in fp32
paged_attention  attention of one new token per request over a paged cache
lora             low-rank adapters of many requests beside a projection
head_norm        the norm of queries or keys for each head
tree_attention   attention of drafted trees' nodes over a paged cache, with tree_masks and tree_seen
verify_tree      which drafted tokens hold, and the token after them
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


def head_norm(x, weight, eps):
    """x [T, heads, dim] -> x / sqrt(mean x^2 + eps) weight, per head."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def tree_masks(parents):
    """Each node's ancestors and itself, as Python integers; a parent of -1 is a root's."""
    got = []
    for i, up in enumerate(parents):
        got.append((got[up] if up >= 0 else 0) | 1 << i)
    return got


def signed64(words):
    return np.array([w - (1 << 64) if w >> 63 else w for w in words], dtype=np.int64)


def tree_seen(length, mask, window=0, sinks=0):
    """Places that a node with this mask sees: cached ones, then nodes."""
    nodes = [length + j for j in range(64) if mask >> j & 1]
    first = max(0, length - max(0, window - len(nodes))) if window else 0
    return [j for j in range(length) if j >= first or j < (sinks if window else 0)] + nodes


def tree_attention(q, k, v, masks, starts, table, lens, scale, window=0, sinks=0):
    """q [T, q_heads, dim] -> (out, lse, bound) in fp64 as paged_attention's; masks are Python integers."""
    T, hq, d = q.shape
    group = hq // k.shape[1]
    page = k.shape[2]
    out, absv = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, top = np.full((T, hq), -np.inf), np.zeros((T, hq))
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        for t in range(starts[b], starts[b + 1]):
            seen = tree_seen(int(lens[b]), masks[t] & ((1 << n) - 1), window, sinks)
            if not seen:
                continue
            at = np.array(seen)
            rows = table[b][at // page], at % page
            for h in range(hq):
                kh, vh = k[rows[0], h // group, rows[1]], v[rows[0], h // group, rows[1]]
                s = scale * (kh @ q[t, h])
                m = s.max()
                p = np.exp(s - m)
                out[t, h] = p @ vh / p.sum()
                lse[t, h] = m + np.log(p.sum())
                top[t, h] = abs(scale) * (np.abs(kh) @ np.abs(q[t, h])).max()
                absv[t, h] = p @ np.abs(vh) / p.sum()
    return out, lse, (top, absv)


def verify_tree(target, draft, tokens, parents, uniform):
    """One request's tree: (path, next). target, draft [n, vocab] in any floats, draft None for chosen tokens. The rest of a refused
    guess is normalised here, step by step."""
    n = len(parents)
    node, path = 0, [0]
    while True:
        p = np.asarray(target[node], dtype=np.float64)
        found = None
        for c in [i for i in range(1, n) if parents[i] == node]:
            x = tokens[c]
            q = np.asarray(draft[node], dtype=np.float64) if draft is not None else np.eye(1, len(p), x)[0]
            if float(uniform[c]) * q[x] < p[x]:
                found = c
                break
            p = np.maximum(p - q, 0)
            if p.sum() > 0:
                p = p / p.sum()
        if found is None:
            break
        node = found
        path.append(node)
    if p.sum() == 0:
        p = np.asarray(target[node], dtype=np.float64)
    sums = np.cumsum(p)
    return path, int(min(np.searchsorted(sums, float(uniform[0]) * sums[-1], side="right"), len(p) - 1))
