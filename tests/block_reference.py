"""Plain float64 implementations of the block-scaled cache's operators, for the tests.

Written from the definitions in include/pa.h, on the CPU, one request at a time; nothing is
shared with the library.
"""

from __future__ import annotations

import math

import torch

CODE_MAX = 448.0


def code_values(codes):
    """float64 values of an e4m3 tensor."""
    return codes.view(torch.uint8).view(torch.float8_e4m3fn).to(torch.float32).double()


def to_code(x):
    """The nearest e4m3 value (ties to even) of finite float64 values, saturated; float64."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-CODE_MAX, CODE_MAX)


def rows(cache, scale, table, n, head):
    """The n positions of one request and kv head, [n, 128] float64."""
    page, block = cache.shape[2], cache.shape[2] // scale.shape[2]
    j = torch.arange(n)
    p = table.long()[j // page]
    x = code_values(cache)[p, head, j % page]
    return x * scale.double()[p, head, j % page // block][:, None]


def attention(q, k_cache, v_cache, k_scale, v_scale, page_table, seqlens, q_lens, sm_scale):
    """(out, lse, sum_j p_j |v_j|, largest s sum_d |q_d k_d| of a row), float64, over the rows of
    every request in order."""
    hq, hkv = q.shape[1], k_cache.shape[1]
    group = hq // hkv
    out, lse, mass, size = [], [], [], []
    at = 0
    for b, (n, d) in enumerate(zip(seqlens, q_lens)):
        o = torch.zeros(d, hq, 128, dtype=torch.float64)
        w = torch.zeros(d, hq, 128, dtype=torch.float64)
        x_max = torch.zeros(d, hq, dtype=torch.float64)
        ls = torch.full((d, hq), -math.inf, dtype=torch.float64)
        for h in range(hkv):
            k = rows(k_cache, k_scale, page_table[b], n, h)
            v = rows(v_cache, v_scale, page_table[b], n, h)
            for i in range(d):
                seen = max(0, n - d + i + 1)
                if seen == 0:
                    continue
                heads = slice(h * group, (h + 1) * group)
                qi = q[at + i, heads].double()
                x = qi @ k[:seen].T * sm_scale
                ls[i, heads] = torch.logsumexp(x, -1)
                p = torch.exp(x - ls[i, heads, None])
                o[i, heads] = p @ v[:seen]
                w[i, heads] = p @ v[:seen].abs()
                x_max[i, heads] = (qi.abs() @ k[:seen].abs().T).amax(-1) * abs(sm_scale)
        out.append(o)
        lse.append(ls)
        mass.append(w)
        size.append(x_max)
        at += d
    return tuple(torch.cat(x) for x in (out, lse, mass, size))


def rope(x, positions, inv_freq, interleaved, amplitude):
    """x [T, heads, 128] -> float64 rows with the first 2 * len(inv_freq) channels turned."""
    y = x.double().clone()
    half = inv_freq.numel()
    turns = torch.tensor([[math.fmod(int(p) * (float(f) / (2 * math.pi)), 1.0) for f in inv_freq]
                          for p in positions], dtype=torch.float64).view(-1, 1, half)
    cos, sin = torch.cos(turns * 2 * math.pi), torch.sin(turns * 2 * math.pi)
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a] = amplitude * (xa * cos - xb * sin)
    y[..., b] = amplitude * (xb * cos + xa * sin)
    return y


def append(values, codes, scale, table, n):
    """One request's new rows (float64 [q_len, Hkv, 128], its newest of n) written to `codes`
    (float64 code values [pages, Hkv, page, 128]) and `scale` (float64), in place."""
    page, block = codes.shape[2], codes.shape[2] // scale.shape[2]
    begin = n - values.shape[0]
    for k in range(begin // block, (n - 1) // block + 1):
        lo, hi = max(k * block, begin), min((k + 1) * block, n)
        p, first = int(table[lo // page]), k * block % page
        i, r = first // block, lo - k * block
        for h in range(codes.shape[1]):
            new = values[lo - begin:hi - begin, h]
            top = float(new.abs().max())
            need = 2.0 ** max(-126, math.ceil(math.log2(top / CODE_MAX))) if top > 0 else 0.0
            old = float(scale[p, h, i])
            to = max(old, need) if r else need
            if r and to != old:
                held = codes[p, h, first:first + r]
                codes[p, h, first:first + r] = to_code(held * (old / to))
            codes[p, h, first + r:first + r + hi - lo] = to_code(new / to) if to > 0 else 0.0
            scale[p, h, i] = to
