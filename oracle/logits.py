"""Logits to probability rows -- oracle, test infrastructure only.

The distribution that verification accepts against ("M7.6 - DeepSeek MTP:
Sequential Modules, Teacher Forcing, and Speculative Runtime" §0x09 takes the
target's row p as given) under one request's sampling parameters: penalties
for tokens already in the text, additive biases, a grammar's set of allowed
tokens, a temperature.  One row at a time, token by token, in fp64.
"""
from __future__ import annotations

import math

import numpy as np

OK, EMPTY, INVALID, INVALID_PARAM = 0, 1, 2, 3


def row(x, prompt, made, repetition=1.0, frequency=0.0, presence=0.0, biases=(), allowed=None, temperature=1.0):
    """(p, status) of one row.  x [V]; prompt and made: token ids before the
    position (made: generated, drafts included); biases: (id, value) pairs of
    which the last of an id holds; allowed [V] bool or None."""
    x = np.asarray(x, dtype=np.float64)
    V = x.shape[0]
    zero = np.zeros(V)
    params = (temperature, repetition, frequency, presence)
    if not all(math.isfinite(v) for v in params) or temperature < 0 or repetition <= 0:
        return zero, INVALID_PARAM
    z = x.copy()
    count = np.zeros(V, dtype=np.int64)
    for v in made:
        if 0 <= v < V:
            count[v] += 1
    seen = set(int(v) for v in list(prompt) + list(made) if 0 <= v < V)
    with np.errstate(over="ignore", invalid="ignore"):
        for v in seen:
            z[v] = z[v] / repetition if z[v] > 0 else z[v] * repetition
            if count[v]:
                z[v] -= frequency * count[v] + presence
        for v, b in dict((int(v), b) for v, b in biases).items():
            if 0 <= v < V:
                z[v] += b
    if allowed is not None:
        z[~np.asarray(allowed, dtype=bool)] = -np.inf
    if np.isnan(z).any() or (z == np.inf).any():
        return zero, INVALID
    m = z.max()
    if m == -np.inf:
        return zero, EMPTY
    if temperature == 0:
        zero[int(np.argmax(z))] = 1.0  # numpy: the lowest index of the maximum
        return zero, OK
    e = np.exp((z - m) / temperature)
    return e / e.sum(), OK


def unpack_mask(words, V):
    """Allowed tokens of one row's mask words (bit v % 32 of word v / 32)."""
    w = np.asarray(words).astype(np.int64) & 0xFFFFFFFF
    return np.array([bool((int(w[v >> 5]) >> (v & 31)) & 1) for v in range(V)])
