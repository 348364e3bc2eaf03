"""Oracle for the 4-bit K/V cache: its layout, the quantising append, the attention.

TEST INFRASTRUCTURE ONLY.  Plain, slow CPU reference in float64; only the tests and the smoke check may import
it.  It shares no code with the CUDA path and imports nothing from the product package.

A value is (c - 8) * s, c a code 0..15, s the scale of its token, KV head and 32 dims (bf16, 5 significant bits); a
(page, KV head) is 18 * dim bytes, K record then V record.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.kv8_oracle import root_path

PAGE, BLOCK = 16, 32
TINY, LARGEST = 2.0 ** -100, 1.3125 * 2.0 ** 123


def bit(e: int) -> int:
    """Bit of code e of the eight of a word."""
    return 16 * (e % 2) + 4 * (e // 2)


def round5(x: float) -> float:
    """x to 5 significant bits, ties to even."""
    if x == 0:
        return 0.0
    unit = 2.0 ** (math.floor(math.log2(abs(x))) - 4)
    return float(np.round(x / unit)) * unit


def quantise(block) -> tuple[np.ndarray, float]:
    """Codes and scale of one block of 32 values (infinities at the end of the range on their side, NaN as 0)."""
    x = np.asarray(block, dtype=np.float64)
    finite = np.where(np.isfinite(x), x, 0.0)
    m = float(finite[np.argmax(np.abs(finite))])
    if abs(m) < TINY:
        return np.full(x.shape, 8), 0.0
    s = round5(m / -8.0)
    s = math.copysign(min(abs(s), LARGEST), s)
    x = np.where(np.isnan(x), 0.0, np.where(np.isinf(x), np.sign(x) * abs(m), x))
    return np.clip(np.round(x / s) + 8, 0, 15).astype(np.int64), s


def bf16_bits(x: float) -> int:
    """Bits of a number that bf16 holds exactly."""
    b = int(np.float32(x).view(np.uint32))
    assert b & 0xFFFF == 0
    return b >> 16


def bf16_value(b: int) -> float:
    return float(np.uint32(int(b) << 16).view(np.float32))


def set_code(record, byte: int, e: int, c: int) -> None:
    """Code e of the word at this byte."""
    at, shift = byte + bit(e) // 8, bit(e) % 8
    record[at] = (int(record[at]) & ~(15 << shift) & 255) | int(c) << shift


def append(cache, k_new, v_new, slots, rows=None):
    """The cache [pages, heads, 2, 9 dim] after the rows have joined; k_new and v_new [rows, heads, dim]."""
    cache = np.array(cache, copy=True)
    heads, dim = cache.shape[1], cache.shape[3] // 9
    nb = dim // BLOCK
    for r, slot in enumerate(int(x) for x in slots):
        if slot < 0:
            continue
        src, page, t = (r if rows is None else int(rows[r])), slot // PAGE, slot % PAGE
        for h in range(heads):
            for is_v, x in enumerate((k_new[src][h], v_new[src][h])):
                rec = cache[page, h, is_v]
                for b in range(nb):
                    codes, s = quantise(x[BLOCK * b:BLOCK * (b + 1)])
                    for i, c in enumerate(codes):
                        if is_v:
                            set_code(rec, (BLOCK * b + i) * 8 + t // 8 * 4, t % 8, c)
                        else:
                            set_code(rec, b * 256 + t * 16 + i // 8 * 4, i % 8, c)
                    at = 8 * dim + 2 * (b * PAGE + t if is_v else t * nb + b)
                    bits = bf16_bits(s)
                    rec[at], rec[at + 1] = bits & 255, bits >> 8
    return cache


def codes_and_scales(cache):
    """K and V codes [pages, heads, 16, dim] and scales [pages, heads, 16, dim / 32] of a cache."""
    cache = np.asarray(cache)
    pages, heads, _, width = cache.shape
    dim = width // 9
    nb = dim // BLOCK
    words = np.ascontiguousarray(cache[..., :8 * dim]).view("<u4").astype(np.uint64)      # [pages, heads, 2, 2 dim]
    codes = np.stack([(words >> np.uint64(bit(e))) & np.uint64(15) for e in range(8)], -1).astype(np.int64)
    k = codes[:, :, 0].reshape(pages, heads, nb, PAGE, 4 * 8).transpose(0, 1, 3, 2, 4).reshape(pages, heads, PAGE, dim)
    v = codes[:, :, 1].reshape(pages, heads, dim, PAGE).transpose(0, 1, 3, 2)
    raw = np.ascontiguousarray(cache[..., 8 * dim:]).view("<u2") & 0xFFF8
    with np.errstate(invalid="ignore"):        # bits that are no number stay none
        scales = (raw.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    sk = scales[:, :, 0].reshape(pages, heads, PAGE, nb)
    sv = scales[:, :, 1].reshape(pages, heads, nb, PAGE).transpose(0, 1, 3, 2)
    return (k, sk), (v, sv)


def values(cache):
    """K and V values [pages, heads, 16, dim] of a cache; scales that are none count as 0."""
    out = []
    for codes, scales in codes_and_scales(cache):
        scales = np.where(np.abs(scales) <= LARGEST, scales, 0.0)        # a NaN is not smaller either
        out.append((codes - 8) * np.repeat(scales, BLOCK, axis=-1))
    return out


def attention(q, cache, k_new, v_new, table, ctx_lens, q_indptr, parents, scale=None, softcap=0.0, slopes=None, window=0,
              only=None):
    """(out [sumN, Hq, D], lse [sumN, Hq], spread [sumN, Hq, D]); spread is the same weighted mean of |v|, the size
    that a relative error of the weights is taken of.  `only`: a set of (row, head) to compute, the rest stay NaN."""
    q, k_new, v_new = (np.asarray(x, dtype=np.float64) for x in (q, k_new, v_new))
    n_rows, hq, dim = q.shape
    group = hq // k_new.shape[1]
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    out, lse = np.full((n_rows, hq, dim), np.nan), np.full((n_rows, hq), np.nan)
    spread = np.full((n_rows, hq, dim), np.nan)
    for b in range(len(q_indptr) - 1):
        lo, hi = int(q_indptr[b]), int(q_indptr[b + 1])
        L, par = int(ctx_lens[b]), [int(x) for x in parents[lo:hi]]
        pages = [int(p) for p in np.asarray(table)[b, :-(-L // PAGE)]]
        held = {}
        for j in range(hi - lo):
            path = root_path(par, j)
            pos = L + len(path) - 1
            seen = [(n, L + d) for d, n in enumerate(path) if not window or L + d > pos - window]
            start = min(L, max(0, pos - window + 1)) if window else 0
            for h in range(hq):
                if only is not None and (lo + j, h) not in only:
                    continue
                g = h // group
                if g not in held:
                    held[g] = [x[:, 0].reshape(-1, dim)[:L] for x in values(np.asarray(cache)[pages, g:g + 1])]
                k = np.concatenate([held[g][0][start:], k_new[[lo + n for n, _ in seen], g]])
                v = np.concatenate([held[g][1][start:], v_new[[lo + n for n, _ in seen], g]])
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
