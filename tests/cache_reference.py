"""Plain float64 implementations of the cache operators, for the tests.

Everything here is written from the definitions in include/pa.h, on the CPU, one request
at a time; nothing is shared with the library or with the attention oracle.
"""

from __future__ import annotations

import math

import torch

NEG_INF = -math.inf


def rope(x, positions, inv_freq, interleaved, amplitude):
    """x [T, heads, 128] -> float64 rows with the first 2 * len(inv_freq) channels turned."""
    y = x.double().clone()
    half = inv_freq.numel()
    # the angle modulo a full turn, from exact integers times the float64 frequency in turns
    turns = torch.tensor([[math.fmod(int(p) * (float(f) / (2 * math.pi)), 1.0) for f in inv_freq]
                          for p in positions], dtype=torch.float64).view(-1, 1, half)
    cos, sin = torch.cos(turns * 2 * math.pi), torch.sin(turns * 2 * math.pi)
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a] = amplitude * (xa * cos - xb * sin)
    y[..., b] = amplitude * (xb * cos + xa * sin)
    return y


def pool_rows(cache, scale, table, n, head):
    """The n positions of one request and kv head, [n, 128] float64."""
    page = cache.shape[2]
    j = torch.arange(n)
    p = table.long()[j // page]
    x = cache[p, head, j % page].double()
    return x if scale is None else x * scale[p, head, j % page].double()[:, None]


def ancestor_rows(parents):
    """Masks of one tree as python integers."""
    rows = []
    for i, up in enumerate(parents):
        rows.append((rows[up] if up >= 0 else 0) | (1 << i))
    return rows


def mask_tensor(rows, words):
    """Integer masks as [len(rows), words] int64."""
    out = torch.zeros((len(rows), words), dtype=torch.int64)
    for r, m in enumerate(rows):
        for w in range(words):
            v = (m >> (64 * w)) & ((1 << 64) - 1)
            out[r, w] = v - (1 << 64) if v >> 63 else v
    return out


def tree_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, seqlens, q_lens, masks,
                   sm_scale):
    """(out, lse, A) float64 with A = softmax . |V| (for tolerances).  masks: a list of
    integers per query row."""
    total, hq, d = q.shape
    hkv = k_cache.shape[1]
    group = hq // hkv
    out = torch.zeros((total, hq, d), dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((total, hq), NEG_INF, dtype=torch.float64)
    at = 0
    for b, (n, ql) in enumerate(zip(seqlens, q_lens)):
        for h in range(hkv):
            k = pool_rows(k_cache, k_scale, page_table[b], n, h)
            v = pool_rows(v_cache, v_scale, page_table[b], n, h)
            for i in range(ql):
                seen = [j for j in range(n) if j < n - ql or (masks[at + i] >> (j - n + ql)) & 1]
                if not seen:
                    continue
                x = (q[at + i, h * group:(h + 1) * group].double() @ k[seen].T) * sm_scale
                total_x = torch.logsumexp(x, -1)
                p = torch.exp(x - total_x[:, None])
                out[at + i, h * group:(h + 1) * group] = p @ v[seen]
                mag[at + i, h * group:(h + 1) * group] = p @ v[seen].abs()
                lse[at + i, h * group:(h + 1) * group] = total_x
        at += ql
    return out, lse, mag


def accumulate(weights, q, lse, k_cache, k_scale, page_table, seqlens, sm_scale):
    """(weights, bound): float64 totals, and the absolute error that fp32 scores allow."""
    w = weights.double().clone()
    bound = 2.0 ** -23 * w.abs()
    hkv, page = k_cache.shape[1], k_cache.shape[2]
    group = q.shape[1] // hkv
    for b, n in enumerate(seqlens):
        j = torch.arange(n)
        p = page_table[b].long()[j // page]
        for h in range(hkv):
            k = pool_rows(k_cache, k_scale, page_table[b], n, h)
            for g in range(h * group, (h + 1) * group):
                if lse[b, g] == NEG_INF:
                    continue
                qd = q[b, g].double()
                x = k @ qd * sm_scale
                add = torch.exp(x - lse[b, g].double())
                # fp32 score: 128 products and 128 sums, each rounded (2^-24); then the
                # factor, lse in base 2, the difference, 2^x (2^-22): all relative to |x|, |lse|
                size = k.abs() @ qd.abs() * sm_scale
                err = 132 * 2.0 ** -24 * size + 2.0 ** -22 * (x.abs() + abs(float(lse[b, g])) + 1)
                w[p, h, j % page] += add
                # e^err - 1 <= 2 err for the small err here; the sums over heads round too
                bound[p, h, j % page] += add * (2 * err + 16 * 2.0 ** -24)
    return w, bound + 2.0 ** -23 * w.abs()


def order_key(w):
    """Sorts like eviction: larger first, NaN before everything, -0 equal to 0."""
    return (0, 0.0) if math.isnan(w) else (1, -w if w != 0 else 0.0)


def kept_positions(w, n, budget, first, recent):
    """Kept positions of one row with weights w[0..n), ascending."""
    if n <= budget:
        return list(range(n))
    always = set(range(first)) | set(range(n - recent, n))
    rest = sorted((j for j in range(n) if j not in always), key=lambda j: (order_key(w[j]), j))
    return sorted(always | set(rest[:budget - first - recent]))


def move(pools, page_table, dst_table, kept, begin):
    """Copies of the pools (each [num_pages, Hkv, page, ...]) with kept[b][h] moved to
    begin[b], begin[b] + 1, ... of dst_table."""
    out = [p.clone() for p in pools]
    page = pools[0].shape[2]
    for b, heads in enumerate(kept):
        for h, rows in enumerate(heads):
            for i, j in enumerate(rows):
                to = begin[b] + i
                src = (int(page_table[b, j // page]), h, j % page)
                dst = (int(dst_table[b, to // page]), h, to % page)
                for old, new in zip(pools, out):
                    new[dst] = old[src]
    return out
