"""Refusals of the 4-bit cache's calls, the rotating append and the log probabilities on the host.  Every call below fails a
host check, so no kernel is launched with the placeholder pointers."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from speculative_decoding_verify_decode_gb300 import build, native
from speculative_decoding_verify_decode_gb300.step import Kv4Cache, Kv4Step

FAKE = 0x10000   # never dereferenced
BAD, UNSUP, WS = native.SD_ERR_INVALID_ARG, native.SD_ERR_UNSUPPORTED, native.SD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def _arrays(layers, ptrs):
    n = max(1, min(layers, 64))
    return [(ctypes.c_void_p * n)(*[None if p is None else p + i * 4096 for i in range(n)]) for p in ptrs]


def _rows(lib, read, layers=1, heads=4, dim=256, page=16, pool=8, ptrs=(FAKE, FAKE << 4, FAKE << 8), stride=0, src=4, slots=FAKE,
          rows=None, max_rows=4, missing=None, odd=None, same=None, off=2):
    arr = _arrays(layers, ptrs)
    if odd is not None:
        arr[odd][0] += off
    if same is not None:
        arr[same[0]][same[1]] = arr[same[2]][same[3]]
    if missing is not None:
        arr[missing] = None
    if read:
        return lib.sd_kv4_read(layers, heads, dim, page, pool, *arr, stride, slots, max_rows, None, None)
    return lib.sd_kv4_append(layers, heads, dim, page, pool, *arr, stride, src, slots, rows, max_rows, None, None)


@pytest.mark.parametrize("read", [False, True], ids=["append", "read"])
@pytest.mark.parametrize("kw,status", [
    (dict(layers=0), BAD), (dict(layers=65), UNSUP), (dict(heads=0), BAD), (dict(heads=65), UNSUP), (dict(dim=64), UNSUP),
    (dict(dim=0), BAD), (dict(page=32), UNSUP), (dict(pool=0), BAD), (dict(pool=1 << 27), UNSUP),
    (dict(ptrs=(None, FAKE, FAKE << 4)), BAD), (dict(ptrs=(FAKE, None, FAKE << 4)), BAD), (dict(ptrs=(FAKE, FAKE << 4, None)), BAD),
    (dict(stride=1023), BAD), (dict(stride=1028), BAD), (dict(stride=-8), BAD), (dict(slots=None), BAD),
    (dict(slots=FAKE + 2), BAD), (dict(max_rows=-1), BAD), *[(dict(missing=i), BAD) for i in range(3)],
    *[(dict(odd=i), BAD) for i in range(3)], *[(dict(odd=i, off=8), BAD) for i in range(3)],
])
def test_rows(lib, read, kw, status):
    assert _rows(lib, read, **kw) == status


def test_append_alone(lib):
    assert _rows(lib, False, src=-1) == BAD and _rows(lib, False, rows=FAKE + 1) == BAD
    assert _rows(lib, False, layers=3, same=(0, 2, 0, 0)) == BAD                     # one cache for two layers


@pytest.mark.parametrize("same", [(1, 0, 2, 0), (1, 1, 1, 0), (2, 2, 2, 0), (1, 2, 2, 0), (1, 1, 0, 2), (2, 0, 0, 0)])
def test_read_refuses_arrays_that_are_written_twice(lib, same):
    assert _rows(lib, True, layers=3, same=same) == BAD


def test_no_rows_are_no_work(lib):
    assert _rows(lib, False, max_rows=0, slots=None) == 0 and _rows(lib, True, max_rows=0, slots=None, ptrs=(FAKE, None, None)) == 0


def _shape(indptr=(0, 5), hq=24, hkv=4, dim=256, max_pages=40, pool=40, **kw):
    s = native.Shape(list(indptr), max_pages, pool, num_q_heads=hq, num_kv_heads=hkv, head_dim=dim)
    for k, v in kw.items():
        setattr(s.c, k, v)
    return s


def _attn(lib, shape=None, opts=None, ws=FAKE, ws_bytes=1 << 40, missing=None, odd=None, off=8, out=FAKE * 2, lse=None):
    ptr = [FAKE] * 7 + [out]
    if missing is not None:
        ptr[missing] = None
    if odd is not None:
        ptr[odd] += off
    shape = shape or _shape()
    return lib.sd_kv4_attn(shape.ref, None if opts is None else ctypes.byref(opts), *ptr, lse, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), BAD), (dict(hkv=0), BAD), (dict(hq=23), BAD), (dict(hq=68, hkv=4), UNSUP), (dict(hq=65, hkv=65), UNSUP),
    (dict(dim=64), UNSUP), (dict(dim=512), UNSUP), (dict(page_size=32), UNSUP), (dict(num_splits=2), UNSUP),
    (dict(num_splits=-1), BAD), (dict(window=-1), BAD), (dict(max_pages=0), BAD), (dict(pool=0), BAD),
    (dict(pool=1 << 27), UNSUP), (dict(batch=0), BAD), (dict(batch=257), UNSUP), (dict(indptr=(0, 65)), UNSUP),
    (dict(indptr=(0, 5, 5)), BAD), (dict(indptr=(1, 5)), BAD), (dict(indptr=()), BAD),
])
def test_attention_shapes(lib, kw, status):
    s = _shape(**kw)
    assert _attn(lib, s) == status
    assert lib.sd_kv4_attn_workspace_size(s.ref) == 0


@pytest.mark.parametrize("kw", [
    *[dict(missing=i) for i in range(8)], *[dict(odd=i) for i in (0, 1, 2, 3, 7)], *[dict(odd=i, off=2) for i in (4, 5, 6)],
    dict(out=FAKE), dict(ws=FAKE + 8), dict(lse=FAKE + 2),
    dict(opts=native.SdKv8Opts(-1.0)), dict(opts=native.SdKv8Opts(float("nan"))), dict(opts=native.SdKv8Opts(0, -2.0)),
    dict(opts=native.SdKv8Opts(0, float("inf"))), dict(opts=native.SdKv8Opts(0, 0, FAKE + 2)),
    dict(opts=native.SdKv8Opts(0, 0, None, 100)), dict(opts=native.SdKv8Opts(0, 0, None, 0, 1020)),
    dict(opts=native.SdKv8Opts(0, 0, None, 0, 0, 1028)), dict(opts=native.SdKv8Opts(0, 0, None, -6144)),
])
def test_attention_arguments(lib, kw):
    assert _attn(lib, **kw) == BAD


def test_attention_caps(lib):
    assert _attn(lib, opts=native.SdKv8Opts(0, 4096.001)) == UNSUP
    assert _attn(lib, opts=native.SdKv8Opts(0, 4096.0), ws=None, ws_bytes=0) == WS       # passes the checks before it


@pytest.mark.parametrize("kw", [dict(), dict(indptr=(0, 1)), dict(indptr=(0, 23)), dict(indptr=(0, 64)), dict(indptr=(0, 20, 84)),
                                dict(indptr=tuple(range(0, 257 * 64, 64))), dict(hq=32, hkv=8, dim=128), dict(hq=64, hkv=64, dim=128),
                                dict(indptr=(0, 31), hq=32, hkv=8, dim=128), dict(hq=16, hkv=1)])
def test_every_valid_shape_needs_a_workspace(lib, kw):
    s = _shape(**kw)
    need = native.sd_kv4_attn_workspace_size(s)
    assert need > 1024
    for opts in (None, native.SdKv8Opts(0, 30.0), native.SdKv8Opts(0, 0, FAKE)):
        assert _attn(lib, s, opts=opts, ws=None, ws_bytes=0) == WS
        assert _attn(lib, s, opts=opts, ws_bytes=need - 1) == WS


# ------------------------------------------------------------------------------------------ rotation

NAMES = ("table", "positions", "q", "k", "v", "q_out", "k_out", "k_cache", "v_cache", "slots")


def _rope(lib, missing=(), same=None, odd=None, off=8, **shape):
    s = dict(num_rows=3, num_q_heads=4, num_kv_heads=2, head_dim=128, rot_dim=64, interleaved=0, table_len=9, page_size=16,
             num_pool_pages=5)
    s.update(shape)
    ptr = {n: FAKE * (i + 1) for i, n in enumerate(NAMES)}
    for n in missing:
        ptr[n] = None
    if same:
        ptr[same[0]] = ptr[same[1]]
    if odd:
        ptr[odd] += off
    return lib.sd_rope_append(ctypes.byref(native.SdRopeShape(**s)), *[ptr[n] for n in NAMES], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_rows=-1), BAD), (dict(num_q_heads=-1), BAD), (dict(num_kv_heads=-1), BAD), (dict(head_dim=0), BAD),
    (dict(rot_dim=0), BAD), (dict(rot_dim=144), BAD), (dict(rot_dim=8), UNSUP), (dict(head_dim=100), UNSUP),
    (dict(head_dim=528, rot_dim=16), UNSUP), (dict(num_q_heads=1025), UNSUP), (dict(interleaved=2), BAD), (dict(table_len=0), BAD),
    (dict(page_size=32), UNSUP), (dict(page_size=0), BAD), (dict(num_pool_pages=0), BAD), (dict(num_pool_pages=1 << 27), UNSUP),
    (dict(q_stride=511), BAD), (dict(q_stride=516), BAD), (dict(k_stride=248), BAD), (dict(v_stride=-8), BAD),
    (dict(q_out_stride=8), BAD), (dict(k_out_stride=260), BAD),
    *[(dict(missing=(n,)), BAD) for n in NAMES if n != "k_out"], (dict(missing=("k_out", "k_cache", "v_cache", "v", "slots")), BAD),
    (dict(num_q_heads=0), BAD), (dict(num_kv_heads=0), BAD), (dict(num_q_heads=0, num_kv_heads=0), BAD),
    *[(dict(odd=n), BAD) for n in NAMES if n not in ("positions", "slots")],
    (dict(odd="positions", off=2), BAD), (dict(odd="slots", off=1), BAD),
    (dict(same=("q_out", "k")), BAD), (dict(same=("q_out", "v")), BAD), (dict(same=("k_out", "q_out")), BAD),
    (dict(same=("k_cache", "v_cache")), BAD), (dict(same=("k_cache", "k")), BAD), (dict(same=("v_cache", "v")), BAD),
    (dict(same=("k_out", "q")), BAD), (dict(same=("q_out", "q"), q_stride=1024), BAD), (dict(same=("k_out", "k"), k_out_stride=512), BAD),
])
def test_rope(lib, kw, status):
    assert _rope(lib, **kw) == status


def test_rope_without_rows_is_no_work(lib):
    assert _rope(lib, missing=NAMES, num_rows=0) == 0


# ------------------------------------------------------------------------------------------ log probabilities

def _lp(lib, rows=700, vocab=1000, dtype=0, logits=FAKE, stride=0, t=1.0, given=1, tokens=FAKE * 2, lp=FAKE * 3, top=4, ids=FAKE * 4,
        top_lp=FAKE * 5, entropy=FAKE * 6, lse=FAKE * 7, ws=FAKE * 8, ws_bytes=1 << 40):
    return lib.sd_logprobs(rows, vocab, dtype, logits, stride, t, given, tokens, lp, top, ids, top_lp, entropy, lse, ws, ws_bytes,
                           None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(vocab=0), BAD), (dict(vocab=(1 << 24) + 1), UNSUP), (dict(dtype=3), BAD), (dict(dtype=-1), BAD),
    (dict(logits=None), BAD), (dict(logits=FAKE + 2), BAD), (dict(logits=FAKE + 1, dtype=1), BAD), (dict(stride=999), BAD),
    (dict(stride=-1000), BAD), (dict(t=0.0), BAD), (dict(t=-1.0), BAD), (dict(t=float("nan")), BAD), (dict(t=float("inf")), BAD),
    (dict(t=1e-39), BAD), (dict(given=-1), BAD), (dict(given=65), UNSUP), (dict(given=0), BAD), (dict(tokens=None), BAD),
    (dict(lp=None), BAD), (dict(top=-1), BAD), (dict(top=33), UNSUP), (dict(top=5, vocab=4), BAD), (dict(top=0), BAD),
    (dict(ids=None), BAD), (dict(top_lp=None), BAD), (dict(entropy=FAKE * 6 + 2), BAD), (dict(lse=FAKE * 6), BAD),
    (dict(lp=FAKE), BAD), (dict(ids=FAKE * 2), BAD), (dict(ws=FAKE * 8 + 8), BAD), (dict(rows=3, vocab=9000, ws=None), WS),
    (dict(rows=3, vocab=9000, ws_bytes=16), WS),
])
def test_logprobs(lib, kw, status):
    assert _lp(lib, **kw) == status


def test_logprobs_workspace(lib):
    for rows, vocab, top in ((1, 151936, 5), (23, 151936, 20), (100, 30000, 32), (1, 5000, 0)):
        need = native.sd_logprobs_workspace_size(rows, vocab, top)
        assert need > 0
        kw = dict(rows=rows, vocab=vocab, top=top, ids=FAKE * 4 if top else None, top_lp=FAKE * 5 if top else None)
        assert _lp(lib, ws_bytes=need - 1, **kw) == WS
    assert native.sd_logprobs_workspace_size(5000, 151936, 20) == 0                  # a row in one piece
    for bad in ((-1, 10, 0), (1, 0, 0), (1, 10, 11), (1, 100, 33), (1, (1 << 24) + 1, 0)):
        assert native.sd_logprobs_workspace_size(*bad) == 0


# ------------------------------------------------------------------------------------------ the binding

def _i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


def _bf(*n):
    return torch.zeros(*n, dtype=torch.bfloat16)


def test_binding_refuses_wrong_cache_tensors():
    cache, new = torch.zeros(8, 4, 2, 9 * 256, dtype=torch.uint8), _bf(6, 4, 256)
    ok = [[cache], [new], [new], _i32(6)]
    for at, t in [(0, [cache.int()]), (0, [cache[..., :-1]]), (0, []), (0, [torch.zeros(8, 4, 16, 128, dtype=torch.uint8)]),
                  (1, [new.float()]), (1, [new[:5]]), (1, [new, new]), (2, [_bf(6, 256, 4).transpose(1, 2)]),
                  (1, [_bf(1, 4, 256).expand(6, 4, 256)]), (3, torch.zeros(6)), (3, _i32(6, 1))]:
        args = list(ok)
        args[at] = t
        with pytest.raises(ValueError):
            native.sd_kv4_append(*args)
        with pytest.raises(ValueError):
            native.sd_kv4_read(args[0], args[3], args[1], args[2])
    with pytest.raises(ValueError):
        native.sd_kv4_read([cache], _i32(5), [new], [new.clone()])
    # one tensor with a leading layer dimension each
    stack, rows = cache[None], new[None]
    for c, k, v in [(stack, rows, rows[:, :5]), (stack, rows[..., None], rows[..., None]), (stack, rows[:, :, :3], rows[:, :, :3]),
                    (stack[..., :-9], rows, rows), (stack, rows.float(), rows.float()), (stack.int(), rows, rows), (stack, new, new),
                    (cache, rows, rows), (stack[:0], rows[:0], rows[:0]), (stack.transpose(1, 2), rows, rows),
                    (stack, rows.transpose(1, 2), rows.transpose(1, 2)), (torch.cat([stack, stack]), rows, rows)]:
        with pytest.raises(ValueError):
            native.sd_kv4_append(c, k, v, _i32(6))
        with pytest.raises(ValueError):
            native.sd_kv4_read(c, _i32(6), k, v)
    with pytest.raises(ValueError, match="CUDA"):
        native.sd_kv4_append(stack, rows, rows, _i32(6))
    with pytest.raises(ValueError, match="CUDA"):
        native.sd_kv4_append(*ok)
    s = _shape((0, 6), pool=8, max_pages=3)
    q = _bf(6, 24, 256)
    ok = [s, q, cache, new, new, _i32(1, 3), _i32(1), _i32(6), torch.empty_like(q)]
    for at, t in [(1, q[:5]), (1, q.half()), (2, cache[:7]), (3, new[:, :3]), (4, _bf(1, 4, 256).expand(6, 4, 256)), (5, _i32(1, 4)),
                  (6, _i32(2)), (7, _i32(5)), (8, q.float())]:
        args = list(ok)
        args[at] = t
        with pytest.raises(ValueError):
            native.sd_kv4_attn(*args)
    with pytest.raises(ValueError):
        native.sd_kv4_attn(*ok, slopes=torch.zeros(23))
    with pytest.raises(ValueError, match="CUDA"):
        native.sd_kv4_attn(*ok)


def test_binding_refuses_wrong_token_tensors():
    table, pos, q, k = torch.zeros(9, 64), _i32(3), _bf(3, 4, 128), _bf(3, 2, 128)
    cache = _bf(5, 2, 16, 128)
    ok = dict(table=table, positions=pos, q=q, k=k, v=k.clone(), q_out=q.clone(), k_out=None, k_cache=cache, v_cache=cache.clone(),
              slots=_i32(3))
    for name, t in [("table", table.double()), ("table", table[:, ::2]), ("table", table[0]), ("positions", pos.long()),
                    ("positions", _i32(3, 1)), ("q", q[0]), ("q", q.float()), ("q_out", _bf(3, 3, 128)), ("k", k[:2]),
                    ("k", _bf(1, 2, 128).expand(3, 2, 128)), ("v", _bf(3, 1, 128)), ("k_cache", _bf(5, 2, 8, 128)),
                    ("v_cache", _bf(4, 2, 16, 128)), ("slots", _i32(2))]:
        with pytest.raises(ValueError):
            native.sd_rope_append(**dict(ok, **{name: t}))
    with pytest.raises(ValueError):
        native.sd_rope_append(table, pos)
    with pytest.raises(ValueError, match="CUDA"):
        native.sd_rope_append(**ok)
    x = torch.zeros(3, 50)
    good = dict(logits=x, tokens=_i32(3, 2), logprobs=torch.zeros(3, 2), top_ids=_i32(3, 4), top_logprobs=torch.zeros(3, 4),
                entropy=torch.zeros(3), lse=torch.zeros(3))
    for name, t in [("logits", x.double()), ("logits", x[0]), ("logits", x.t()), ("logits", torch.zeros(1, 50).expand(3, 50)),
                    ("tokens", _i32(2, 2)), ("tokens", torch.zeros(3, 2)), ("logprobs", torch.zeros(3, 1)), ("top_ids", _i32(4, 4)),
                    ("top_logprobs", torch.zeros(3, 5)), ("entropy", torch.zeros(4)), ("lse", torch.zeros(3, 1))]:
        with pytest.raises(ValueError):
            native.sd_logprobs(**dict(good, **{name: t}))
    with pytest.raises(ValueError, match="CUDA"):
        native.sd_logprobs(**good)


def test_cache_and_step_hold_what_the_calls_need():
    c = Kv4Cache(2, 5, 12, 3, num_kv_heads=2, head_dim=128, device="cpu")
    assert c.kv.shape == (3, 12, 2, 2, 1152) and c.kv.dtype == torch.uint8 and c.free_list.tolist() == list(range(11, -1, -1))
    s = Kv4Step(c, [0, 3, 7], 1000, num_q_heads=8, top=5)
    assert s.out.shape == (3, 7, 8, 128) and s.top_ids.shape == (7, 5) and s.q_turned.shape == (3, 7, 8, 128)
    for top in (-1, 33):
        with pytest.raises(ValueError):
            Kv4Step(c, [0, 3, 7], 1000, num_q_heads=8, top=top)
    with pytest.raises(ValueError):
        Kv4Step(c, [0, 3, 7], 4, num_q_heads=8, top=5)
    assert s.k_turned.shape == (3, 7, 2, 128) and s.attn_ws.numel() == native.sd_kv4_attn_workspace_size(s.shape)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_struct_and_constants_match_the_headers(tmp_path):
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    names = [f[0] for f in native.SdRopeShape._fields_]
    offs = " ".join(f'printf(" %zu", offsetof(sd_rope_shape, {n}));' for n in names)
    bits = ["SD_DEV_NOT_FINITE", "SD_DEV_BAD_POSITION"]
    more = " ".join(f'printf(" %d", {b});' for b in bits) + ' printf(" %d", SD_KV4_MAX_SCALE == 1.3125 * 0x1p123);'
    src = tmp_path / "a.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "sd_kv4.h"\n#include "sd_rope.h"\n#include "sd_logprobs.h"\n'
                   f'int main(void) {{ printf("%zu", sizeof(sd_rope_shape)); {offs} {more}'
                   ' printf(" %d %d %d %d", SD_LOGITS_F32, SD_LOGITS_BF16, SD_LOGITS_F16, SD_LOGPROBS_MAX_TOP); return 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-I", inc, str(src), "-o", str(tmp_path / "a")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(native.SdRopeShape)] + [getattr(native.SdRopeShape, n).offset for n in names] + \
        [getattr(native, b) for b in bits] + [1, 0, 1, 2, native.SD_LOGPROBS_MAX_TOP]
