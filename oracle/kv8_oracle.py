"""Oracle for the 8-bit block-scaled K/V cache: page tables and slot maps, the quantising append, the attention.

TEST INFRASTRUCTURE ONLY.  Plain, slow CPU reference in float64; only the tests and the smoke check may import
it.  It shares no code with the CUDA path and imports nothing from the product package.

A page holds 16 tokens of every KV head as e4m3 codes; a code stands for decode(code) * scale of its (page, head).
"""
from __future__ import annotations

import math

import numpy as np

from oracle.fp8_oracle import E4M3_MAX, e4m3_decode, e4m3_encode

PAGE = 16
MIN_EXP, MAX_EXP = -100, 100
VALUES = np.array([e4m3_decode(c) for c in range(256)], dtype=np.float64)
_FINITE = VALUES[:127]


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 codes of float64 values: ties to the even code, saturation, NaN -> 0x7F (elementwise e4m3_encode)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    up = np.clip(np.searchsorted(_FINITE, np.where(np.isnan(a), 0.0, a)), 0, 126)     # first finite value >= a
    down = np.maximum(up - 1, 0)
    mid = (_FINITE[up] + _FINITE[down]) / 2
    code = np.where((a < mid) | ((a == mid) & (down % 2 == 0)), down, up)
    code = np.where(a >= E4M3_MAX, 126, code) | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def block_exp(amax: float) -> int:
    """Exponent of the smallest power of two s with amax <= 448 s, clamped."""
    if amax <= 0:
        return MIN_EXP
    e = math.floor(math.log2(amax)) - 10
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return max(MIN_EXP, min(MAX_EXP, e))


def append(codes, scales, new, slots, rows=None):
    """New (codes, scales) of one layer and tensor: [pages, heads, 16, dim] uint8 and [pages, heads]."""
    codes, scales = np.array(codes, copy=True), np.array(scales, dtype=np.float64, copy=True)
    groups: dict[int, list[tuple[int, int]]] = {}
    for r, s in enumerate(int(x) for x in slots):
        if s >= 0:
            groups.setdefault(s // PAGE, []).append((s % PAGE, r if rows is None else int(rows[r])))
    for page, items in groups.items():
        first = min(t for t, _ in items)
        for h in range(codes.shape[1]):
            x = np.stack([np.asarray(new[src][h], dtype=np.float64) for _, src in items])
            fin = np.abs(x[np.isfinite(x)])
            s = 2.0 ** block_exp(float(fin.max()) if fin.size else 0.0)
            if first > 0:
                old = scales[page, h]
                s = max(s, old)
                if s != old:
                    codes[page, h, :first] = encode(VALUES[codes[page, h, :first]] * (old / s))
            scales[page, h] = s
            for (t, _), row in zip(items, x):
                codes[page, h, t] = encode(row / s)
    return codes, scales


def dequantise(codes, scales):
    return VALUES[np.asarray(codes)] * np.asarray(scales, dtype=np.float64)[:, :, None, None]


def root_path(parents, j):
    path = [j]
    while parents[path[-1]] >= 0:
        path.append(int(parents[path[-1]]))
    return path[::-1]


def attention(q, k_codes, v_codes, k_scales, v_scales, k_new, v_new, table, ctx_lens, q_indptr, parents, scale=None,
              softcap=0.0, slopes=None, window=0, only=None):
    """(out [sumN, Hq, D], lse [sumN, Hq], spread [sumN, Hq, D]); spread is the same weighted mean of |v|, the size
    that a relative error of the weights is taken of.  `only`: a set of (row, head) to compute, the rest stay NaN."""
    q, k_new, v_new = (np.asarray(x, dtype=np.float64) for x in (q, k_new, v_new))
    n_rows, hq, dim = q.shape
    hkv = k_new.shape[1]
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    out, lse = np.full((n_rows, hq, dim), np.nan), np.full((n_rows, hq), np.nan)
    spread = np.full((n_rows, hq, dim), np.nan)
    for b in range(len(q_indptr) - 1):
        lo, hi = int(q_indptr[b]), int(q_indptr[b + 1])
        L, par = int(ctx_lens[b]), [int(x) for x in parents[lo:hi]]
        pages = [int(p) for p in np.asarray(table)[b, :-(-L // PAGE)]]
        ctx = {}
        for j in range(hi - lo):
            path = root_path(par, j)
            pos = L + len(path) - 1
            first = max(0, pos - window + 1) if window else 0
            seen = [(n, L + d) for d, n in enumerate(path) if not window or L + d > pos - window]
            for h in range(hq):
                if only is not None and (lo + j, h) not in only:
                    continue
                g = h // (hq // hkv)
                if g not in ctx:
                    rows = lambda c, s: (VALUES[np.asarray(c)[pages, g]] * np.asarray(s, dtype=np.float64)[pages, g]
                                         [:, None, None]).reshape(-1, dim)[:L]
                    ctx[g] = (rows(k_codes, k_scales), rows(v_codes, v_scales))
                start = min(first, L)
                k = np.concatenate([ctx[g][0][start:], k_new[[lo + n for n, _ in seen], g]])
                v = np.concatenate([ctx[g][1][start:], v_new[[lo + n for n, _ in seen], g]])
                at = np.concatenate([np.arange(start, L), [p for _, p in seen]])
                s = k @ q[lo + j, h] * scale
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s + float(slopes[h]) * (at - pos)
                m = s.max()
                w = np.exp(s - m)
                out[lo + j, h] = w @ v / w.sum()
                spread[lo + j, h] = w @ np.abs(v) / w.sum()
                lse[lo + j, h] = m + math.log(w.sum())
    return out, lse, spread


def pages_extend(ctx, add, table, held, free, max_rows, q_indptr=None, path=None):
    """(table, held, free list, slots, rows, row_indptr, ctx) after the call; ``free`` is a list used as a stack."""
    table, held, free = np.array(table, copy=True), [int(x) for x in held], [int(x) for x in free]
    slots, rows, indptr = [], [], [0]
    for b, (c, a) in enumerate(zip(ctx, add)):
        while held[b] * PAGE < c + a:
            table[b, held[b]] = free.pop()
            held[b] += 1
        for i in range(int(a)):
            pos = int(c) + i
            slots.append(int(table[b, pos // PAGE]) * PAGE + pos % PAGE)
            rows.append(len(rows) if path is None else int(q_indptr[b]) + int(path[b][i]))
        indptr.append(len(slots))
    pad = [-1] * (max_rows - len(slots))
    return table, held, free, slots + pad, rows + pad, indptr, [int(c) + int(a) for c, a in zip(ctx, add)]


def pages_release(keep, table, held, free):
    """(held, free list) after the call."""
    held, free = [int(x) for x in held], [int(x) for x in free]
    for b, n in enumerate(keep):
        left = min(held[b], -(-int(n) // PAGE))
        free += [int(p) for p in np.asarray(table)[b, left:held[b]]]
        held[b] = left
    return held, free


__all__ = ["VALUES", "encode", "block_exp", "append", "dequantise", "attention", "pages_extend", "pages_release",
           "e4m3_encode"]
