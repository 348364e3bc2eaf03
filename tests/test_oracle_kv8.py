"""Pins of the block-scaled cache's oracle: the format, the block scale, append, attention, page tables."""
import math

import numpy as np
import pytest

import oracle.kv8_oracle as kv8
from oracle.fp8_oracle import e4m3_encode


def test_encode_is_the_scalar_rounding():
    rng = np.random.default_rng(0)
    mids = (kv8.VALUES[1:126] + kv8.VALUES[:125]) / 2
    x = np.concatenate([rng.normal(size=3000) * 2.0 ** rng.integers(-14, 10, 3000), mids, -mids, kv8.VALUES[:127],
                        [448, 449, 464, 1e9, -1e9, np.inf, -np.inf, 0.0, -0.0, 2.0 ** -10, -2.0 ** -10, np.nan]])
    assert [int(c) for c in kv8.encode(x)] == [e4m3_encode(v) for v in x]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (1.75, -8), (1.0, -8), (1.76, -7), (0.0, -100),
                                    (1e-45, -100), (3e38, 100), (448 * 2.0 ** -100, -100), (449 * 2.0 ** 99, 100)])
def test_block_exp(amax, e):
    assert kv8.block_exp(amax) == e


def test_append_begins_and_continues_pages():
    rng = np.random.default_rng(1)
    codes, scales = np.full((4, 2, 16, 8), 0x55, np.uint8), np.full((4, 2), 0.5)
    x = rng.normal(size=(20, 2, 8))
    slots = [2 * 16 + 13, 2 * 16 + 14, 2 * 16 + 15] + [16 + i for i in range(16)] + [-1]
    got, s = kv8.append(codes, scales, x, slots)
    assert np.array_equal(got[[0, 3]], codes[[0, 3]]) and np.array_equal(s[[0, 3]], scales[[0, 3]])
    assert np.all(s[2] == 0.5) and np.array_equal(got[2, :, :13], codes[2, :, :13])    # the old scale is the larger
    assert np.all(np.abs(kv8.VALUES[got[1]]).max(axis=(1, 2)) > 224)                   # a fresh page uses the range
    back = kv8.dequantise(got, s)
    assert np.abs(back[1].transpose(1, 0, 2) - x[3:19]).max() <= 2.0 ** -4 * np.abs(x).max()
    # larger values behind small ones: the scale grows and the old values stay what they were, to a rounding
    big, s2 = kv8.append(got, s, 640 * x[:1], [2 * 16 + 15])
    assert np.all(s2[2] > 0.5)
    old, new = kv8.dequantise(got, s)[2, :, :15], kv8.dequantise(big, s2)[2, :, :15]
    assert np.all(np.abs(old - new) <= 2.0 ** -10 * s2[2][:, None, None])


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    hkv, dim = 2, 8
    codes = kv8.encode(rng.normal(size=(3, hkv, 16, dim)) * 50)
    scales = 2.0 ** rng.integers(-8, -5, (3, hkv)).astype(float)
    table = np.array([[2, 0, -1]])
    kn, vn = rng.normal(size=(3, hkv, dim)), rng.normal(size=(3, hkv, dim))
    zero = np.zeros((3, 4, dim))
    par = [-1, 0, 0]
    out, lse, _ = kv8.attention(zero, codes, codes, scales, scales, kn, vn, table, [19], [0, 3], par)
    v = kv8.dequantise(codes, scales)
    ctx = np.concatenate([v[2], v[0][:, :3]], 1)                       # [heads, 19, dim]
    for h in range(4):
        want = (ctx[h // 2].sum(0) + vn[0, h // 2] + vn[2, h // 2]) / 21   # node 2: root and itself
        np.testing.assert_allclose(out[2, h], want, rtol=1e-12)
        assert abs(lse[2, h] - math.log(21)) < 1e-12
    # window 1: every node sees itself alone; a huge bias leaves the nearest key alone too
    one, l1, _ = kv8.attention(rng.normal(size=(3, 4, dim)), codes, codes, scales, scales, kn, vn, table, [19], [0, 3],
                               par, window=1)
    np.testing.assert_allclose(one, np.repeat(vn, 2, axis=1), rtol=1e-12)
    far, _, _ = kv8.attention(zero, codes, codes, scales, scales, kn, vn, table, [19], [0, 3], par, slopes=[1e4] * 4)
    np.testing.assert_allclose(far, np.repeat(vn, 2, axis=1), rtol=1e-12)
    # a cap far above every score changes nothing, a tiny one makes all scores alike
    q = rng.normal(size=(3, 4, dim))
    base = kv8.attention(q, codes, codes, scales, scales, kn, vn, table, [19], [0, 3], par)[0]
    np.testing.assert_allclose(kv8.attention(q, codes, codes, scales, scales, kn, vn, table, [19], [0, 3], par,
                                             softcap=1e7)[0], base, rtol=1e-9)
    np.testing.assert_allclose(kv8.attention(q, codes, codes, scales, scales, kn, vn, table, [19], [0, 3], par,
                                             softcap=1e-9)[0], out, rtol=1e-6)


def test_pages_extend_and_release_round_trip():
    table = np.full((3, 5), -1)
    free = list(range(10, 22))
    t, held, left, slots, rows, ind, ctx = kv8.pages_extend([0, 0, 0], [17, 0, 40], table, [0, 0, 0], free, 60)
    assert held == [2, 0, 3] and ind == [0, 17, 17, 57] and ctx == [17, 0, 40]
    assert list(t[0, :2]) == [21, 20] and slots[16] == 20 * 16 and slots[57:] == [-1] * 3 and rows[:57] == list(range(57))
    held2, back = kv8.pages_release([16, 0, 0], t, held, left)
    assert held2 == [1, 0, 0] and sorted(back) == sorted(set(free) - {21})
