"""Pins of the 4-bit cache's oracle: the format by hand, by exhaustive search and by the layout's definition; the attention
against closed forms, torch's softmax attention and the 8-bit oracle."""
import math

import numpy as np
import pytest
import torch

import oracle.kv4_oracle as kv4
import oracle.kv8_oracle as kv8


@pytest.mark.parametrize("x,want", [(1.0, 1.0), (-3.0, -3.0), (31.0, 31.0), (33.0, 32.0), (35.0, 36.0), (33.5, 34.0), (0.0, 0.0),
                                    (2.0 ** -40 * 31, 2.0 ** -40 * 31), (63.5, 64.0), (-33.0, -32.0)])
def test_five_significant_bits(x, want):
    assert kv4.round5(x) == want


def test_blocks_by_hand():
    x = np.zeros(32)
    x[3], x[4], x[5], x[6] = 8.0, -8.0, 4.5, -4.5           # the largest, first: 8 -> s = -1; ties of rint go to even
    codes, s = kv4.quantise(x)
    assert s == -1.0 and codes[3] == 0 and codes[4] == 15 and codes[0] == 8
    assert codes[5] == 4 and codes[6] == 12                  # 4.5 / -1 = -4.5 -> -4
    x[3], x[4] = -8.0, 8.0
    codes, s = kv4.quantise(x)
    assert s == 1.0 and codes[3] == 0 and codes[4] == 15     # -8 s is a code, +8 s is held as 7 s
    assert kv4.quantise(np.full(32, 2.0 ** -101))[1] == 0.0 and (kv4.quantise(np.full(32, 2.0 ** -101))[0] == 8).all()
    x[:] = 1.0
    x[0], x[1], x[2] = math.inf, -math.inf, math.nan
    codes, s = kv4.quantise(x)
    assert s == -0.125 and list(codes[:4]) == [0, 15, 8, 0]


def test_every_code_is_the_nearest_value():
    rng = np.random.default_rng(1)
    for _ in range(300):
        x = torch.from_numpy(rng.normal(size=32) * 2.0 ** rng.integers(-20, 20)).bfloat16().double().numpy()
        codes, s = kv4.quantise(x)
        grid = (np.arange(16) - 8) * s
        best = np.abs(grid[None] - x[:, None]).min(axis=1)
        np.testing.assert_array_equal(np.abs(grid[codes] - x), best)
        m = x[np.argmax(np.abs(x))]
        assert abs(s * -8 - m) <= abs(m) * 2.0 ** -5 and np.float32(s).view(np.uint32) & 0x7FFFF == 0


def test_values_are_bf16():
    """(c - 8) s of a 5-bit s is a bf16 number."""
    for m in range(16, 32):
        for c in range(16):
            v = (c - 8) * m * 2.0 ** -9
            assert float(torch.tensor(v).bfloat16()) == v


def test_layout_round_trip():
    rng = np.random.default_rng(2)
    k, v = (torch.from_numpy(rng.normal(size=(20, 3, 128))).bfloat16().double().numpy() for _ in "kv")
    slots = list(range(5, 16)) + list(range(32, 41))
    before = rng.integers(0, 256, (3, 3, 2, 9 * 128), dtype=np.uint8)
    cache = kv4.append(before, k, v, slots)
    (ck, sk), (cv, sv) = kv4.codes_and_scales(cache)
    for r, slot in enumerate(slots):
        for codes, scales, x in ((ck, sk, k), (cv, sv, v)):
            for h in range(3):
                for b in range(4):
                    want, s = kv4.quantise(x[r, h, 32 * b:32 * b + 32])
                    assert scales[slot // 16, h, slot % 16, b] == s
                    np.testing.assert_array_equal(codes[slot // 16, h, slot % 16, 32 * b:32 * b + 32], want)
    # one code moves one nibble, at the bit that the layout names
    again = np.array(cache, copy=True)
    word = again[0, 1, 0, 2 * 256 + 7 * 16 + 3 * 4:][:4].view("<u4")     # K, block 2, token 7, dims 88..95
    word ^= np.uint32(15 << kv4.bit(5))
    (c2, _), _ = kv4.codes_and_scales(again)
    where = np.argwhere(c2 != ck)
    assert [tuple(x) for x in where] == [(0, 1, 7, 64 + 3 * 8 + 5)]
    # what got no row stays
    (b1, _), (b2, _) = kv4.codes_and_scales(before)
    np.testing.assert_array_equal(ck[1], b1[1])
    np.testing.assert_array_equal(cv[0, :, :5], b2[0, :, :5])


def _case(seed, ctx, parents, hq=4, hkv=2, dim=128):
    rng = np.random.default_rng(seed)
    bf = lambda *s: torch.from_numpy(rng.normal(size=s)).bfloat16().double().numpy()
    pages = -(-ctx // 16)
    table = rng.permutation(pages + 2)[:max(1, pages)][None]
    rows = bf(ctx, hkv, dim), bf(ctx, hkv, dim)
    slots = [int(table[0, t // 16]) * 16 + t % 16 for t in range(ctx)]
    cache = kv4.append(np.zeros((pages + 2, hkv, 2, 9 * dim), np.uint8), *rows, slots)
    n = len(parents)
    return dict(q=bf(n, hq, dim), cache=cache, k_new=bf(n, hkv, dim), v_new=bf(n, hkv, dim), table=table, ctx_lens=[ctx],
                q_indptr=[0, n], parents=parents)


def test_attention_equals_torch_on_the_values():
    c = _case(3, 37, [-1, 0, 1, 2])
    out, lse, spread = kv4.attention(**c)
    k, v = (x[c["table"][0]].transpose(0, 2, 1, 3).reshape(-1, 2, 128)[:37] for x in kv4.values(c["cache"]))
    k, v = np.concatenate([k, c["k_new"]]), np.concatenate([v, c["v_new"]])
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).transpose(0, 1)[None]
    mask = torch.ones(4, 41, dtype=torch.bool).tril(37)
    want = torch.nn.functional.scaled_dot_product_attention(t(c["q"]), t(k.repeat(2, axis=1)), t(v.repeat(2, axis=1)), attn_mask=mask)
    np.testing.assert_allclose(out, want[0].transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)
    assert (spread + 1e-15 >= np.abs(out)).all()


@pytest.mark.parametrize("kw", [dict(), dict(window=9), dict(softcap=3.0), dict(slopes=[0.5, 0.1, 0.0, 0.3]), dict(scale=0.4)])
def test_attention_equals_the_8_bit_oracle_on_values_that_both_hold(kw):
    """Whole numbers -8 .. 7 are codes here and e4m3 values there."""
    rng = np.random.default_rng(5)
    c = _case(4, 50, [-1, 0, 0, 2, 1])
    codes8 = {}
    for i, x in enumerate("kv"):
        n = rng.integers(-8, 8, (6, 2, 16, 128)).astype(np.float64)
        n[..., ::32] = -8                                        # so that every scale is 1
        codes8[x] = kv8.encode(n)
        rows = n.transpose(0, 2, 1, 3).reshape(-1, 2, 128)
        c["cache"] = kv4.append(c["cache"], rows if i == 0 else kept, rows, range(96)) if i else c["cache"]
        kept = rows
    assert c["cache"].shape[0] == 6
    one = np.ones((6, 2))
    got = kv4.attention(**c, **kw)
    want = kv8.attention(c["q"], codes8["k"], codes8["v"], one, one, c["k_new"], c["v_new"], c["table"], c["ctx_lens"],
                         c["q_indptr"], c["parents"], **kw)
    for g, w in zip(got, want):
        np.testing.assert_allclose(g, w, rtol=1e-12, atol=1e-12)
