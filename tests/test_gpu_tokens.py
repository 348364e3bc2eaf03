"""The rotating append and the log probabilities on the GPU, through the C ABI, against the float64 oracle.

Rotation: a turned value is x_a c - x_b s of bf16 and fp32 factors.  Off by 2^-8 of the result (rounding to bf16) plus 3 fp32
roundings, 3 * 2^-24 (|x_a| + |x_b|); copied values are exact.

Log probabilities, with d2 = (x - m) / T in base 2: a term e^d is off by 2^-22 (ex2) + |d2| 2^-23 (rounding of d2 and of the
factor log2 e / T), sums by 2^-21 of themselves (16 terms a tile and thread in a row, then trees), so log S by
e_s = 2^-21 + (2^-22 + D 2^-23) r, where r = rest / S <= 1 is the share of the terms beside the largest and D = 64 bounds |d2|
where terms count; relative to rest when rest is small, so the error of log S is at most e_s min(1, rest).  A log probability
adds 2 * 2^-23 of the difference's size, |x_t - m| / T; the entropy adds 2^-20 of W / S, whose terms carry one more rounding.
"""
import math

import numpy as np
import pytest
import torch

import oracle.token_oracle as tok
from speculative_decoding_verify_decode_gb300 import native

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def np64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def table_of(length, rot, theta=1e6):
    angle = np.arange(length)[:, None] * theta ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()


def near_rotated(got, x, table, pos, inter):
    got, x, table = np64(got), np64(x), np64(table)
    want = tok.rotate(x, table, pos, inter)
    half = table.shape[1] // 2
    mate = np.abs(x).copy()
    a = np.arange(0, 2 * half, 2) if inter else np.arange(half)
    b = a + 1 if inter else a + half
    mate[..., a] = mate[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    bound = 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -24 * mate
    bound[..., 2 * half:] = 0
    assert np.all(np.abs(got - want) <= bound), (np.abs(got - want) - bound).max()


@pytest.mark.parametrize("rows,hq,hkv,dim,rot,inter", [
    (1, 24, 4, 256, 256, False), (5, 24, 4, 256, 64, False), (40, 32, 8, 128, 128, True), (33, 7, 1, 96, 48, False),
    (3, 2, 2, 16, 16, True), (3, 2, 2, 16, 16, False), (700, 4, 2, 64, 32, True), (9, 64, 64, 512, 512, False), (2, 3, 5, 48, 16, False),
])
def test_rotation_and_append_match_oracle(rows, hq, hkv, dim, rot, inter):
    rng = np.random.default_rng(rows + dim)
    pool = rows // 16 + 3
    table = table_of(200, rot)
    pos = rng.integers(0, 200, rows)
    slots = rng.permutation(pool * 16)[:rows]
    pos[0] = 199
    if rows > 4:
        pos[2], slots[3] = -1, -1                                    # padding; a row that is turned but not kept
    mk = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).bfloat16().cuda()
    q, k, v, kc, vc = mk(rows, hq, dim), mk(rows, hkv, dim), mk(rows, hkv, dim), mk(pool, hkv, 16, dim), mk(pool, hkv, 16, dim)
    kc0, vc0 = kc.clone(), vc.clone()
    q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    status = i32([0])
    native.sd_rope_append(table, i32(pos.tolist()), q, k, v, q_out, k_out, kc, vc, i32(slots.tolist()), inter, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    on = pos >= 0
    near_rotated(q_out[torch.from_numpy(on)], q[torch.from_numpy(on)], table, pos[on], inter)
    near_rotated(k_out[torch.from_numpy(on)], k[torch.from_numpy(on)], table, pos[on], inter)
    assert torch.all(q_out[torch.from_numpy(~on)] == 7.0) and torch.all(k_out[torch.from_numpy(~on)] == 7.0)
    kept = np.where(on, slots, -1)
    np.testing.assert_array_equal(np64(kc), tok.put(np64(kc0), np64(k_out), kept))
    np.testing.assert_array_equal(np64(vc), tok.put(np64(vc0), np64(v), kept))


def test_rotation_of_a_fused_projection_and_in_place():
    rng = np.random.default_rng(1)
    qkv = torch.from_numpy(rng.normal(size=(50, 32 + 16, 128)).astype(np.float32)).bfloat16().cuda()
    table, pos = table_of(64, 128), i32(rng.integers(0, 64, 50).tolist())
    q, k = qkv[:, :32], qkv[:, 32:40]
    q_out, k_out = torch.empty(50, 32, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(50, 8, 128, dtype=torch.bfloat16, device="cuda")
    native.sd_rope_append(table, pos, q, k, q_out=q_out, k_out=k_out)
    near_rotated(q_out, q, table, pos.tolist(), False)
    near_rotated(k_out, k, table, pos.tolist(), False)
    rest = qkv[:, 40:].clone()
    native.sd_rope_append(table, pos, q, k, q_out=q, k_out=k)
    assert torch.equal(q, q_out) and torch.equal(k, k_out) and torch.equal(qkv[:, 40:], rest)
    # queries alone, keys alone
    native.sd_rope_append(table, pos, qkv[:, :32], q_out=q_out)
    near_rotated(q_out, q, table, pos.tolist(), False)
    native.sd_rope_append(table, pos, k=k, k_out=k_out, interleaved=True)
    near_rotated(k_out, k, table, pos.tolist(), True)


def test_rotation_reports_bad_positions_and_slots():
    table = table_of(10, 32)
    mk = lambda *s: torch.randn(*s, device="cuda").bfloat16()
    q, k, v, kc, vc = mk(5, 2, 64), mk(5, 1, 64), mk(5, 1, 64), mk(2, 1, 16, 64), mk(2, 1, 16, 64)
    kc0 = kc.clone()
    q_out, status = torch.full_like(q, 7.0), i32([0])
    native.sd_rope_append(table, i32([0, 10, -2, 3, -1]), q, k, v, q_out, None, kc, vc, i32([-1, 1, 2, 32, 5]), False, status)
    assert int(status) == native.SD_DEV_BAD_POSITION | native.SD_DEV_BAD_SLOT
    assert torch.equal(kc, kc0)
    near_rotated(q_out[[0, 3]], q[[0, 3]], table, [0, 3], False)
    assert torch.all(q_out[[1, 2, 4]] == 7.0)
    status.zero_()
    native.sd_rope_append(table, i32([4] * 5), q, k, v, q_out, None, kc, vc, i32([-2, -1, -1, -1, -1]), False, status)
    assert int(status) == native.SD_DEV_BAD_SLOT and torch.equal(kc, kc0)


def test_no_rows():
    table = table_of(10, 32)
    e = lambda h: torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda")
    native.sd_rope_append(table, i32([]), e(2), e(1), q_out=e(2), k_out=e(1))
    native.sd_logprobs(torch.empty(0, 50, device="cuda"), entropy=torch.empty(0, device="cuda"))
    torch.cuda.synchronize()


def test_a_cache_beyond_32_bit_offsets():
    pool = 140000                                                     # 32 KB a page and tensor
    kc, vc = (torch.empty(pool, 4, 16, 256, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    assert kc.numel() > 2 ** 31
    table = table_of(10, 256)
    mk = lambda *s: torch.randn(*s, device="cuda").bfloat16()
    k, v, k_out = mk(2, 4, 256), mk(2, 4, 256), mk(2, 4, 256)
    native.sd_rope_append(table, i32([3, 9]), k=k, v=v, k_out=k_out, k_cache=kc, v_cache=vc, slots=i32([pool * 16 - 1, pool * 16 - 9]))
    near_rotated(k_out, k, table, [3, 9], False)
    assert torch.equal(kc[-1, :, 15], k_out[0]) and torch.equal(vc[-1, :, 7], v[1])


# ------------------------------------------------------------------------------------------ log probabilities

def run(logits, tokens=None, top=0, temperature=1.0, dtype=torch.float32, ws=None):
    x = logits.to(dtype).cuda() if not logits.is_cuda else logits
    rows, vocab = x.shape
    out = dict(entropy=torch.full((rows,), 7.0, device="cuda"), lse=torch.full((rows,), 7.0, device="cuda"))
    if tokens is not None:
        out["tokens"], out["logprobs"] = tokens.int().cuda(), torch.full(tokens.shape, 7.0, device="cuda")
    if top:
        out["top_ids"] = torch.full((rows, top), 7, dtype=torch.int32, device="cuda")
        out["top_logprobs"] = torch.full((rows, top), 7.0, device="cuda")
    status = i32([0])
    need = native.sd_logprobs_workspace_size(rows, vocab, top)
    native.sd_logprobs(x, temperature=temperature, workspace=torch.full((max(16, need),), 0xFF, dtype=torch.uint8, device="cuda"),
                       dev_status=status, **out)
    torch.cuda.synchronize()
    return x, out, int(status)


def check(x, out, rows=None, temperature=1.0):
    top = out["top_ids"].shape[1] if "top_ids" in out else 0
    for r in range(x.shape[0]) if rows is None else rows:
        row = np64(x[r])
        toks = out["tokens"][r].tolist() if "tokens" in out else []
        given, ids, best, entropy, lse = tok.logprobs(row, toks, top, temperature)
        m = row.max() / temperature
        log_s = lse - m
        rest = math.expm1(-best[0]) if top else math.expm1(log_s)
        share = rest / (1 + rest)
        e_s = (2.0 ** -21 + (2.0 ** -22 + 64 * 2.0 ** -23) * 1.0) * min(1.0, rest) if rest < 1 else \
            2.0 ** -21 + (2.0 ** -22 + 64 * 2.0 ** -23) * share
        e_s += 2.0 ** -22 * abs(log_s)
        size = lambda v: 2 * 2.0 ** -23 * abs(v) + e_s
        f32 = lambda v: float(np.float64(v).astype(np.float32))      # a difference beyond fp32's 3.4e38 is an infinity there
        if "tokens" in out:
            for g, w in zip(out["logprobs"][r].tolist(), given):
                assert g == f32(w) or abs(g - w) <= size(w), (r, g, w)
        if top:
            assert out["top_ids"][r].tolist() == ids
            for g, w in zip(out["top_logprobs"][r].tolist(), best):
                assert g == f32(w) or abs(g - w) <= size(w), (r, g, w)
        # W / S = entropy - log S: its terms have the sums' errors and d's own
        w_s = abs(entropy - max(log_s, 0.0))
        e_h = e_s + w_s * (2.0 ** -20 + 64 * 2.0 ** -23 + 2.0 ** -21)
        assert abs(float(out["entropy"][r]) - entropy) <= e_h, (r, float(out["entropy"][r]), entropy, e_h)
        assert abs(float(out["lse"][r]) - lse) <= e_s + 2.0 ** -22 * (abs(lse) + abs(m)), (r, float(out["lse"][r]), lse)


def model_rows(seed, rows, vocab, peak=12.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * 2.5
    x.scatter_(1, torch.randint(vocab, (rows, 2), generator=g), torch.rand(rows, 2, generator=g) * peak + 4)
    return x, torch.randint(-1, vocab, (rows, 3), generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab,top,temperature", [
    (1, 1, 1, 1.0), (3, 7, 7, 1.0), (2, 64, 32, 0.5), (5, 1001, 5, 1.0), (4, 4096, 20, 1.3), (3, 4097, 32, 1.0),
    (2, 50257, 20, 0.7), (1, 151936, 5, 1.0), (3, 151936, 0, 1.0), (9, 20000, 1, 2.0), (700, 300, 4, 1.0),
])
def test_logprobs_match_oracle(rows, vocab, top, temperature, dtype):
    x, t = model_rows(rows + vocab, rows, vocab)
    x, out, status = run(x, t, top, temperature, dtype)
    assert status == 0
    check(x, out, range(rows) if rows < 20 else range(0, rows, 97), temperature)


def test_many_rows_of_a_large_vocabulary():
    """Rows in one piece each, over many tiles: the list is cut again and again."""
    x, t = model_rows(3, 640, 30011)
    x, out, status = run(x, t, 32, 1.0, torch.bfloat16)
    assert status == 0
    check(x, out, (0, 1, 319, 639))


@pytest.mark.parametrize("kind", ["rising", "falling", "constant", "two_values", "one_warp", "zeros_of_both_signs", "mostly_masked",
                                  "nearly_certain", "certain", "far_apart"])
@pytest.mark.parametrize("rows,vocab", [(1, 9000), (620, 9000)])
def test_rows_where_selection_and_sums_can_go_wrong(kind, rows, vocab):
    v = torch.arange(vocab)
    row = {
        "rising": v * 2.0 ** -9, "falling": -v * 2.0 ** -9, "constant": torch.full((vocab,), 3.5),
        "two_values": (v % 3 == 0).float(), "one_warp": ((v % 1024) < 32).float() * (1 + v % 5),
        "zeros_of_both_signs": torch.where(v % 2 == 0, -0.0, 0.0), "mostly_masked": torch.where(v % 1000 == 7, v * 2.0 ** -10, -math.inf),
        "nearly_certain": torch.where(v == 4000, 30.0, 0.0), "certain": torch.where(v == 4000, 1e4, -1e4),
        "far_apart": torch.where(v % 2 == 0, 3e38, -3e38),
    }[kind].float()
    for top in (1, 32):
        x, out, status = run(row[None].repeat(rows, 1), torch.tensor([[0, 4000, vocab - 1, vocab, -1]]).repeat(rows, 1), top)
        assert status == 0
        check(x, out, (0, rows - 1))


def test_rows_of_nothing_and_rows_that_are_none():
    x = torch.zeros(5, 6000)
    x[0] = -math.inf
    x[1, 5] = math.nan
    x[2, 5999] = math.inf
    x[3, 17] = -math.inf
    _, out, status = run(x, torch.tensor([[17, -1]] * 5), 4)
    assert status == native.SD_DEV_NAN_LOGITS
    inf = math.inf
    assert float(out["lse"][0]) == -inf and float(out["entropy"][0]) == 0.0
    assert out["logprobs"][0].tolist() == [-inf, -inf] and out["top_ids"][0].tolist() == [0, 1, 2, 3]
    assert out["top_logprobs"][0].tolist() == [-inf] * 4
    for r in (1, 2):
        assert all(math.isnan(v) for v in [float(out["lse"][r]), float(out["entropy"][r])] + out["logprobs"][r].tolist() +
                   out["top_logprobs"][r].tolist())
        assert out["top_ids"][r].tolist() == [-1] * 4
    assert out["logprobs"][3].tolist() == [-inf, -inf]
    check(x.cuda(), out, (3, 4))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_rows_that_lie_apart_and_off_their_alignment(dtype):
    x, t = model_rows(8, 6, 5003)
    wide = torch.full((6, 5011), math.nan, dtype=dtype, device="cuda")
    part = wide[:, 3:5006]
    part.copy_(x)
    _, out, status = run(part, t, 20)
    assert status == 0
    check(part, out)


def test_logprobs_are_the_same_bits_every_time_and_in_a_graph():
    x, t = model_rows(9, 23, 151936)
    x, first, _ = run(x, t, 20)
    for _ in range(5):
        _, out, _ = run(x, t, 20)
        assert all(torch.equal(out[k], first[k]) for k in first)
    ws = torch.empty(native.sd_logprobs_workspace_size(23, 151936, 20), dtype=torch.uint8, device="cuda")
    out = {k: torch.zeros_like(v) if k != "tokens" else v for k, v in first.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        native.sd_logprobs(x, workspace=ws, **out)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], first[k]) for k in first)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_long_rows_where_the_set_is_hard_to_find(dtype):
    """Rows that one CTA works through alone: sorted, alike, few values, masked, a late rise."""
    rows, vocab, top = 1830, 41001, 32
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(rows, vocab, generator=gen).mul_(3).to(dtype)
    ramp = torch.linspace(-20, 20, vocab)
    some = {0: ramp, 1: -ramp, 2: torch.full((vocab,), 1.5), 3: (torch.arange(vocab) % 3).float(), 4: torch.full((vocab,), -math.inf),
            5: torch.where(torch.arange(vocab) > vocab - 20, 1.0, -math.inf), 6: torch.cat([torch.zeros(vocab - 5), torch.full((5,), 40.0)]),
            7: torch.where(torch.arange(vocab) % 512 == 511, 2.0, 0.0), 8: torch.where(torch.arange(vocab) // 512 == 40, 2.0, 0.0),
            9: torch.full((vocab,), torch.finfo(dtype).min), 10: torch.cat([torch.full((vocab - 40,), torch.finfo(dtype).min), torch.zeros(40)])}
    for r, v in some.items():
        x[r] = v.to(dtype)
        x[rows - 1 - r] = v.to(dtype)
    x, out, status = run(x, tokens=torch.randint(vocab, (rows, 3), generator=gen), top=top, dtype=dtype)
    assert status == 0
    check(x, out, rows=[r for r in some if r != 4] + [rows - 1, rows - 9, 100, 900, 1500])
    for r in (4, rows - 5):        # nothing but -infinity: exact
        assert float(out["entropy"][r]) == 0.0 and float(out["lse"][r]) == -math.inf and out["top_ids"][r].tolist() == list(range(top))
        assert torch.all(out["logprobs"][r] == -math.inf) and torch.all(out["top_logprobs"][r] == -math.inf)


@pytest.mark.parametrize("dtype,size,temperature", [(torch.float16, 1.0, 1000.0), (torch.float16, 20.0, 60.0), (torch.float16, 1.0, 100.0),
                                                    (torch.bfloat16, 1e4, 1e-3), (torch.float32, 3e6, 1.0), (torch.float32, 1.0, 1e30),
                                                    (torch.float32, 1e30, 1e30), (torch.bfloat16, 1e35, 1e36)])
@pytest.mark.parametrize("rows", [1, 700])
def test_scales_of_logits_and_temperatures(rows, dtype, size, temperature):
    """Where the exponents' shift is large, or the type has nothing far enough below the maximum; masked tokens count nothing."""
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(rows, 9001, generator=gen)
    x[:, 100:4000] = -math.inf
    x[0, 8000] = 6.0
    x[rows - 1, 9000] = 7.0
    x, out, status = run((x * size).to(dtype), tokens=torch.randint(9001, (rows, 4), generator=gen), top=7, temperature=temperature, dtype=dtype)
    assert status == 0
    check(x, out, rows=[0, rows - 1, rows // 2], temperature=temperature)


@pytest.mark.parametrize("rows,vocab,top", [(160, (1 << 21) + 5, 20), (1, (1 << 24) - 3, 32), (1, 1 << 24, 0), (200, 1, 1), (3, 31, 31)])
def test_the_largest_and_smallest_vocabularies(rows, vocab, top):
    """Rows in one piece of more than 4096 segments, the most logits there can be, and next to none."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 3).bfloat16()
    tokens = torch.randint(vocab, (rows, 2), generator=gen, device="cuda")
    out = run(x, tokens=tokens, top=top)[1]
    for r in {0, rows // 2, rows - 1}:
        z = x[r].double()
        lse = torch.logsumexp(z, 0)
        # sums: 2^-21, and the exponentials 2^-22 + 64 * 2^-23 (see the head of this file); the logarithm and the difference fp32
        tol = 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -17 + 2.0 ** -22 * (float(lse.abs()) + float(z.abs().max()))
        assert abs(float(out["lse"][r]) - float(lse)) <= tol
        assert torch.all((out["logprobs"][r].double() - (z[tokens[r]] - lse)).abs() <= tol)
        p = (z - lse).exp()
        h = -float((p * (z - lse)).sum())
        assert abs(float(out["entropy"][r]) - h) <= tol + h * (2.0 ** -20 + 2.0 ** -17)
        if top:
            order = torch.sort(x[r].float(), descending=True, stable=True)[1][:top]
            assert torch.equal(out["top_ids"][r].long(), order)
            assert torch.all((out["top_logprobs"][r].double() - (z[order] - lse)).abs() <= tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab", [(200, 20008), (200, 20001), (6, 20008)])
def test_one_value_that_is_none_anywhere(rows, vocab, dtype):
    """A NaN of either sign or a +infinity at any place of a row makes that row none, and no other; values behind the last row
    and between rows that lie apart are not looked at."""
    gen = torch.Generator().manual_seed(rows)
    wide = torch.full((rows, vocab + 24), math.nan)
    wide[:, :vocab] = torch.randn(rows, vocab, generator=gen) * 4
    wide[:, 7] = -math.inf
    bad = {r: [math.nan, -math.nan, math.inf][r % 3] for r in range(0, rows, 2)}
    where = {r: (r * 997 + 3) % vocab if 0 < r < rows - 2 else (0 if r == 0 else vocab - 1) for r in bad}
    for r, v in bad.items():
        wide[r, where[r]] = v
    x = wide.to(dtype).cuda()[:, :vocab]
    tokens = torch.tensor([[7, 1 + r] for r in range(rows)])
    x, out, status = run(x, tokens, 6, dtype=dtype)
    assert status == native.SD_DEV_NAN_LOGITS
    for r in bad:
        values = torch.cat([out["lse"][r:r + 1], out["entropy"][r:r + 1], out["logprobs"][r], out["top_logprobs"][r]])
        assert torch.isnan(values).all() and torch.all(out["top_ids"][r] == -1), r
    good = [r for r in range(rows) if r not in bad]
    assert torch.isfinite(out["lse"][good]).all() and torch.isfinite(out["entropy"][good]).all()
    assert torch.all(out["logprobs"][good, 0] == -math.inf)
    check(x, out, rows=good[:2] + good[-2:])


@pytest.mark.parametrize("top", [1, 7, 31, 32])
@pytest.mark.parametrize("vocab", [512, 700, 4600, 8500, 32000])
@pytest.mark.parametrize("kind", ["normal", "rising", "falling", "two", "steps"])
def test_alternatives_of_pieces_that_end_inside_a_segment(kind, vocab, top):
    """The set and its order, where the last piece of a row has a few warps' logits only, and where many logits are equal."""
    gen = torch.Generator().manual_seed(vocab + top)
    x = torch.randn(3, vocab, generator=gen) * 4
    if kind in ("rising", "falling"):
        x = torch.sort(x, 1, descending=kind == "falling")[0]
    elif kind == "two":
        x = (x > 3).float()
    elif kind == "steps":
        x = torch.floor(torch.sort(x, 1)[0] * 2)
    for dtype in (torch.float32, torch.float16):
        y, out, status = run(x.to(dtype), top=top, dtype=dtype)
        assert status == 0
        order = torch.sort(y.float(), dim=1, descending=True, stable=True)[1][:, :top]
        assert torch.equal(out["top_ids"].long(), order)
