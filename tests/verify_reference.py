"""Plain implementation of the draft verification, for the tests: the definition in include/pa.h
with Python's integers and 64-bit floats, one request at a time, nothing shared with the library."""

from __future__ import annotations

import math

import numpy as np

UNITS = 2 ** 42


def units(w):
    """floor(2^42 min(w, 1)) of float32 weights, as Python-exact int64."""
    return np.floor(np.minimum(w.astype(np.float64), 1.0) * UNITS).astype(np.int64)


def left_over(p, q, c):
    """max(p - c q, 0), rounded once to float32."""
    if c == 0:
        return p
    exact = p.astype(np.longdouble) - np.longdouble(c) * q.astype(np.longdouble)
    return np.maximum(exact.astype(np.float32), np.float32(0))


def draw(w, u):
    """First index whose prefix sum passes floor(u T), or None where nothing is there."""
    total = np.cumsum(units(w))
    if total[-1] == 0:
        return None
    t = min(math.floor(float(np.float32(u)) * float(total[-1])), int(total[-1]) - 1)
    return int(np.searchsorted(total, t, side="right"))


def verify(target, draft, tokens, parents, uniforms, final):
    """(accepted rows, next token or None) of one request; target and draft [rows, vocab] float32
    (draft None: proposed for certain)."""
    vocab = target.shape[1]
    node, path = 0, [0]
    c, s, left, gone = np.float32(0), np.float32(1), 1.0, []
    for i in range(1, len(tokens)):
        if parents[i] != node:
            continue
        x, u = tokens[i], float(np.float32(uniforms[i]))
        inside = 0 <= x < vocab
        if draft is not None:
            if s is None:
                total = int(units(left_over(target[node], draft[node], c)).sum())
                s = np.float32(np.float32(total) * np.float32(2.0 ** -42))
            w = left_over(target[node], draft[node], c)[x] if inside else np.float32(0)
            q = draft[node][x] if inside else np.float32(1)
            ok = u * float(q) * float(s) < float(w)
            if not ok:
                c, s = np.float32(c + s), None
        else:
            w = target[node][x] if inside and x not in gone else np.float32(0)
            ok = u * left < float(w)
            if not ok and w > 0:
                gone.append(x)
                left -= float(w)
        if ok:
            node = i
            path.append(i)
            c, s, left, gone = np.float32(0), np.float32(1), 1.0, []
    w = left_over(target[node], draft[node], c).copy() if draft is not None else target[node].copy()
    w[gone] = 0
    token = draw(w, final)
    if token is None:
        token = draw(target[node], final)
    return path, token
