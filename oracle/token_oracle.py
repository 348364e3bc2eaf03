"""Oracle for the calls around a step's tokens: the rotating append, and log probabilities with entropy and alternatives.

TEST INFRASTRUCTURE ONLY.  Plain, slow CPU reference in float64; only the tests may import it.  It shares no code with
the CUDA path and imports nothing from the product package.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 16


def rotate(x, table, positions, interleaved=False):
    """x [rows, heads, dim] turned: pair i by the angle whose cosine and sine are table[p][i] and table[p][rot / 2 + i]."""
    y = np.array(x, dtype=np.float64, copy=True)
    half = np.shape(table)[1] // 2
    for r, p in enumerate(int(p) for p in positions):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
            z = (y[r, :, a] + 1j * y[r, :, b]) * (float(table[p][i]) + 1j * float(table[p][half + i]))
            y[r, :, a], y[r, :, b] = z.real, z.imag
    return y


def put(cache, rows, slots):
    """A paged cache [pages, heads, 16, dim] with rows set at their slots."""
    cache = np.array(cache, copy=True)
    for row, s in zip(rows, (int(s) for s in slots)):
        if s >= 0:
            cache[s // PAGE, :, s % PAGE] = row
    return cache


def logprobs(logits, tokens, top, temperature=1.0):
    """(logprobs, top_ids, top_logprobs, entropy, lse) of one row, by python's own float sums."""
    x = [float(v) for v in logits]
    z = [v / temperature for v in x]
    m = max(z)
    if m == -math.inf:
        return [-math.inf] * len(tokens), list(range(top)), [-math.inf] * top, 0.0, -math.inf
    # the largest term is 1 and stands apart, so what the rest adds to it keeps its digits
    at = z.index(m)
    rest = math.fsum(math.exp(v - m) for i, v in enumerate(z) if i != at)
    log_sum = math.log1p(rest)
    entropy = log_sum - math.fsum(math.exp(v - m) * (v - m) for v in z if v > -math.inf) / (1 + rest)
    lp = lambda v: v - m - log_sum
    ids = sorted(range(len(x)), key=lambda i: (-x[i], i))[:top]
    given = [lp(z[t]) if 0 <= t < len(x) else -math.inf for t in tokens]
    return given, ids, [lp(z[i]) for i in ids], entropy, m + log_sum
