"""Refusals of the block-scaled cache's calls on the host.  Every call below fails a host check, so no kernel is
launched with the placeholder pointers."""
import ctypes

import pytest
import torch

from speculative_decoding_verify_decode_gb300 import build, native

FAKE = 0x10000   # never dereferenced
BAD, UNSUP, WS = native.SD_ERR_INVALID_ARG, native.SD_ERR_UNSUPPORTED, native.SD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def _extend(lib, batch=2, max_pages=8, pool=64, ctx=FAKE, add=FAKE + 64, indptr=None, path=None, max_path=0,
            table=FAKE + 128, held=FAKE + 192, new_held=FAKE + 256, free=FAKE + 320, count=FAKE + 384,
            new_count=FAKE + 448, max_rows=10, slots=FAKE + 512, rows=None, row_indptr=None, new_ctx=None):
    ind = None if indptr is None else (ctypes.c_int * len(indptr))(*indptr)
    return lib.sd_pages_extend(batch, max_pages, pool, ctx, add, ind, path, max_path, table, held, new_held, free, count,
                               new_count, max_rows, slots, rows, row_indptr, new_ctx, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), BAD), (dict(batch=native.MAX_BATCH + 1), UNSUP), (dict(max_pages=0), BAD), (dict(pool=0), BAD),
    (dict(max_pages=(1 << 26) + 1), UNSUP), (dict(pool=1 << 27), UNSUP), (dict(max_rows=-1), BAD),
    (dict(ctx=None), BAD), (dict(add=None), BAD), (dict(table=None), BAD), (dict(held=None), BAD),
    (dict(new_held=None), BAD), (dict(free=None), BAD), (dict(count=None), BAD), (dict(new_count=None), BAD),
    (dict(slots=None), BAD),
    (dict(indptr=[0, 3, 5]), BAD), (dict(path=FAKE + 600, max_path=4), BAD),                # one without the other
    (dict(indptr=[0, 3, 5], path=FAKE + 600, max_path=0), BAD),
    (dict(indptr=[1, 3, 5], path=FAKE + 600, max_path=4), BAD), (dict(indptr=[0, 3, 68], path=FAKE + 600, max_path=4), UNSUP),
    (dict(new_held=FAKE + 192), BAD), (dict(new_count=FAKE + 384), BAD), (dict(new_ctx=FAKE), BAD),   # aliases
    (dict(new_held=FAKE), BAD), (dict(rows=FAKE + 64), BAD),
    (dict(ctx=FAKE + 2), BAD), (dict(table=FAKE + 129), BAD), (dict(slots=FAKE + 514), BAD), (dict(rows=FAKE + 701), BAD),
])
def test_pages_extend(lib, kw, status):
    assert _extend(lib, **kw) == status


def _release(lib, batch=2, max_pages=8, pool=64, keep=FAKE, table=FAKE + 64, held=FAKE + 128, new_held=FAKE + 192,
             free=FAKE + 256, count=FAKE + 320, new_count=FAKE + 384):
    return lib.sd_pages_release(batch, max_pages, pool, keep, table, held, new_held, free, count, new_count, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), BAD), (dict(batch=257), UNSUP), (dict(pool=0), BAD), (dict(keep=None), BAD), (dict(table=None), BAD),
    (dict(held=None), BAD), (dict(new_held=None), BAD), (dict(free=None), BAD), (dict(count=None), BAD),
    (dict(new_count=None), BAD), (dict(new_held=FAKE + 128), BAD), (dict(new_count=FAKE + 320), BAD),
    (dict(new_count=FAKE + 128), BAD), (dict(free=FAKE + 64), BAD), (dict(held=FAKE + 130), BAD), (dict(free=FAKE + 257), BAD),
])
def test_pages_release(lib, kw, status):
    assert _release(lib, **kw) == status


def _append(lib, layers=1, heads=4, dim=256, page=16, pool=8, ptr=FAKE, stride=0, src=4, slots=FAKE, max_rows=4,
            missing=None, odd=None):
    arr = [(ctypes.c_void_p * max(1, min(layers, 64)))(*[ptr] * max(1, min(layers, 64))) for _ in range(6)]
    if odd is not None:
        arr[odd][0] = FAKE + 2
    if missing is not None:
        arr[missing] = None
    return lib.sd_kv8_append(layers, heads, dim, page, pool, *arr, stride, src, slots, None, max_rows, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(layers=0), BAD), (dict(layers=65), UNSUP), (dict(heads=0), BAD), (dict(heads=65), UNSUP), (dict(dim=64), UNSUP),
    (dict(dim=0), BAD), (dict(page=32), UNSUP), (dict(pool=0), BAD), (dict(pool=1 << 27), UNSUP), (dict(ptr=None), BAD),
    (dict(ptr=FAKE + 4), BAD), (dict(stride=1023), BAD), (dict(stride=1028), BAD), (dict(stride=-8), BAD),
    (dict(src=-1), BAD), (dict(slots=None), BAD), (dict(slots=FAKE + 2), BAD), (dict(max_rows=-1), BAD),
    *[(dict(missing=i), BAD) for i in range(6)], *[(dict(odd=i), BAD) for i in range(6)],
])
def test_append(lib, kw, status):
    assert _append(lib, **kw) == status


def _shape(indptr=(0, 5), hq=24, hkv=4, dim=256, max_pages=40, pool=40, **kw):
    s = native.Shape(list(indptr), max_pages, pool, num_q_heads=hq, num_kv_heads=hkv, head_dim=dim)
    for k, v in kw.items():
        setattr(s.c, k, v)
    return s


def _attn(lib, shape=None, opts=None, ws=FAKE, ws_bytes=1 << 40, missing=None, odd=None, off=8, out=FAKE * 2):
    ptr = [FAKE] * 10 + [out]
    if missing is not None:
        ptr[missing] = None
    if odd is not None:
        ptr[odd] += off
    shape = shape or _shape()
    return lib.sd_kv8_attn(shape.ref, None if opts is None else ctypes.byref(opts), *ptr, None, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), BAD), (dict(hkv=0), BAD), (dict(hq=23), BAD), (dict(hq=68, hkv=4), UNSUP), (dict(hq=65, hkv=65), UNSUP),
    (dict(dim=64), UNSUP), (dict(dim=512), UNSUP), (dict(page_size=32), UNSUP), (dict(num_splits=2), UNSUP),
    (dict(num_splits=-1), BAD), (dict(window=-1), BAD), (dict(max_pages=0), BAD), (dict(pool=0), BAD),
    (dict(pool=1 << 27), UNSUP), (dict(batch=0), BAD), (dict(batch=257), UNSUP), (dict(indptr=(0, 65)), UNSUP),
    (dict(indptr=(0, 5, 5)), BAD), (dict(indptr=(1, 5)), BAD),
])
def test_attention_shapes(lib, kw, status):
    s = _shape(**kw)
    assert _attn(lib, s) == status
    assert lib.sd_kv8_attn_workspace_size(s.ref) == 0


@pytest.mark.parametrize("kw", [
    *[dict(missing=i) for i in range(11)], *[dict(odd=i) for i in (0, 1, 2, 5, 6, 10)],
    *[dict(odd=i, off=2) for i in (3, 4, 7, 8, 9)], dict(out=FAKE), dict(ws=FAKE + 8),
    dict(opts=native.SdKv8Opts(-1.0)), dict(opts=native.SdKv8Opts(float("nan"))), dict(opts=native.SdKv8Opts(0, -2.0)),
    dict(opts=native.SdKv8Opts(0, float("inf"))), dict(opts=native.SdKv8Opts(0, 0, FAKE + 2)),
    dict(opts=native.SdKv8Opts(0, 0, None, 100)), dict(opts=native.SdKv8Opts(0, 0, None, 0, 1020)),
    dict(opts=native.SdKv8Opts(0, 0, None, 0, 0, 1028)), dict(opts=native.SdKv8Opts(0, 0, None, -6144)),
])
def test_attention_arguments(lib, kw):
    assert _attn(lib, **kw) == BAD


def test_attention_workspace(lib):
    s = _shape((0, 23), max_pages=2050, pool=2050)
    need = native.sd_kv8_attn_workspace_size(s)
    if need:
        assert _attn(lib, s, ws=None, ws_bytes=0) == WS
        assert _attn(lib, s, ws_bytes=need - 1) == WS


def test_binding_refuses_wrong_tensors():
    """Types, shapes, strides and devices are checked before the library is called."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    good = dict(ctx_lens=i32(2), add_lens=i32(2), page_table=i32(2, 4), held=i32(2), new_held=i32(2), free_list=i32(9),
                free_count=i32(1), new_free_count=i32(1), slots=i32(5))
    for name, t in [("ctx_lens", i32(3)), ("held", torch.zeros(2)), ("page_table", i32(2, 8)[:, ::2]),
                    ("free_count", i32(2)), ("slots", torch.zeros(5, dtype=torch.int64))]:
        with pytest.raises(ValueError):
            native.sd_pages_extend(**dict(good, **{name: t}))
    with pytest.raises(ValueError):
        native.sd_pages_extend(**good, path=i32(2, 3), q_indptr=[0, 3])          # a q_indptr of another batch
    with pytest.raises(ValueError, match="CUDA"):
        native.sd_pages_extend(**good)                                            # host tensors
    codes, scales = torch.zeros(8, 4, 16, 256, dtype=torch.uint8), torch.zeros(8, 4)
    new = torch.zeros(6, 4, 256, dtype=torch.bfloat16)
    ok = [[codes], [codes], [scales], [scales], [new], [new], i32(6)]
    for at, t in [(0, [codes.int()]), (2, [scales[:, :3]]), (4, [new.float()]), (4, [new[:5]]), (1, [codes, codes]),
                  (5, [torch.zeros(6, 256, 4, dtype=torch.bfloat16).transpose(1, 2)])]:
        args = list(ok)
        args[at] = t
        with pytest.raises(ValueError):
            native.sd_kv8_append(*args)
    s = _shape((0, 6), pool=8, max_pages=3)
    q = torch.zeros(6, 24, 256, dtype=torch.bfloat16)
    ok = [s, q, codes, codes, scales, scales, new, new, i32(1, 3), i32(1), i32(6), torch.empty_like(q)]
    for at, t in [(1, q[:5]), (1, q.half()), (2, codes[:7]), (4, scales.double()), (8, i32(1, 4)), (9, i32(2)),
                  (10, i32(5)), (11, q.float())]:
        args = list(ok)
        args[at] = t
        with pytest.raises(ValueError):
            native.sd_kv8_attn(*args)
    with pytest.raises(ValueError):
        native.sd_kv8_attn(*ok, slopes=torch.zeros(23))


def test_structs_and_constants_match_the_header():
    """The option struct's mirror and the status bits, as a C compiler has them."""
    import os
    import shutil
    import subprocess
    import tempfile
    if shutil.which("gcc") is None:
        pytest.skip("needs a C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    names = [f[0] for f in native.SdKv8Opts._fields_]
    offs = " ".join(f'printf(" %zu", offsetof(sd_kv8_opts, {n}));' for n in names)
    bits = ["SD_DEV_NO_PAGES", "SD_DEV_BAD_SCALE", "SD_DEV_BAD_SLOT"]
    more = " ".join(f'printf(" %d", {b});' for b in bits)
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "a.c")
        with open(src, "w") as f:
            f.write('#include <stddef.h>\n#include <stdio.h>\n#include "sd_kv8.h"\n'
                    f'int main(void) {{ printf("%zu", sizeof(sd_kv8_opts)); {offs} {more} return 0; }}\n')
        subprocess.run(["gcc", "-std=c11", "-I", inc, src, "-o", os.path.join(d, "a")], check=True)
        got = [int(x) for x in subprocess.run([os.path.join(d, "a")], check=True, capture_output=True,
                                              text=True).stdout.split()]
    assert got == [ctypes.sizeof(native.SdKv8Opts)] + [getattr(native.SdKv8Opts, n).offset for n in names] + \
        [getattr(native, b) for b in bits]


def test_binding_refuses_rows_that_overlap():
    """Rows expanded from one have stride 0, which means dense to the library: it would read behind the tensor."""
    codes, scales = torch.zeros(8, 4, 16, 256, dtype=torch.uint8), torch.zeros(8, 4)
    one = lambda heads, layers=(): torch.zeros(*layers, 1, heads, 256, dtype=torch.bfloat16)
    new, broad = torch.zeros(6, 4, 256, dtype=torch.bfloat16), one(4).expand(6, 4, 256)
    rows = torch.zeros(6, dtype=torch.int32)
    shifted = torch.zeros(8 * 512, dtype=torch.bfloat16).as_strided((6, 4, 256), (512, 256, 1))   # half a row apart
    for k, v in [([broad], [broad]), ([broad], [new]), ([new], [broad]), ([shifted], [shifted]),
                 (one(4, (1,)).expand(1, 6, 4, 256),) * 2]:
        with pytest.raises(ValueError, match="rows overlap"):
            native.sd_kv8_append([codes], [codes], [scales], [scales], k, v, rows)
    two = one(4, (2,)).expand(2, 6, 4, 256)
    with pytest.raises(ValueError, match="rows overlap"):
        native.sd_kv8_append([codes] * 2, [codes] * 2, [scales] * 2, [scales] * 2, two, two, rows)
    s = _shape((0, 6), pool=8, max_pages=3)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    q = torch.zeros(6, 24, 256, dtype=torch.bfloat16)
    ok = [s, q, codes, codes, scales, scales, new, new, i32(1, 3), i32(1), i32(6), torch.empty_like(q)]
    for at, t in [(1, one(24).expand(6, 24, 256)), (6, broad), (7, broad), (7, shifted)]:
        args = list(ok)
        args[at] = t
        with pytest.raises(ValueError, match="rows overlap"):
            native.sd_kv8_attn(*args)
    # one head a row, and one row, have no such stride to check
    narrow = _shape((0, 6), hq=1, hkv=1, pool=8, max_pages=3)
    args = [narrow, one(1).expand(6, 1, 256), codes[:, :1].contiguous(), codes[:, :1].contiguous(), scales[:, :1].contiguous(),
            scales[:, :1].contiguous(), new[:, 0:1].contiguous(), new[:, 0:1].contiguous(), i32(1, 3), i32(1), i32(6),
            torch.empty(6, 1, 256, dtype=torch.bfloat16)]
    with pytest.raises(ValueError, match="rows overlap"):
        native.sd_kv8_attn(*args)
    args[1] = torch.zeros(6, 3, 256, dtype=torch.bfloat16)[:, 1:2]                  # rows that lie apart pass
    with pytest.raises(ValueError, match="CUDA"):
        native.sd_kv8_attn(*args)


def test_score_caps_beyond_what_the_formula_keeps(lib):
    """c - 2 c / (1 + exp(2 x / c)) loses c 2^-22 of a score: 1 % of the weights at 1e5, everything at 1e7."""
    for cap in (4096.001, 1e5, 1e7, 1e30, 3.4e38):
        assert _attn(lib, opts=native.SdKv8Opts(0, cap)) == UNSUP
    assert _attn(lib, opts=native.SdKv8Opts(0, 4096.0), ws=None, ws_bytes=0) == WS       # passes the checks before it


@pytest.mark.parametrize("kw", [dict(), dict(indptr=(0, 1)), dict(indptr=(0, 23)), dict(indptr=(0, 64)), dict(indptr=(0, 20, 84)),
                                dict(indptr=tuple(range(0, 257 * 64, 64))), dict(hq=32, hkv=8, dim=128),
                                dict(indptr=(0, 31), hq=32, hkv=8, dim=128), dict(hq=64, hkv=64, dim=128), dict(hq=16, hkv=1)])
def test_every_valid_shape_needs_a_workspace(lib, kw):
    """Never 0, and a byte less is refused, for plain, capped and biased scores (their plans differ beyond 96 columns)."""
    s = _shape(**kw)
    need = native.sd_kv8_attn_workspace_size(s)
    assert need > 1024
    for opts in (None, native.SdKv8Opts(0, 30.0), native.SdKv8Opts(0, 0, FAKE)):
        assert _attn(lib, s, opts=opts, ws=None, ws_bytes=0) == WS
        assert _attn(lib, s, opts=opts, ws_bytes=need - 1) == WS


def test_an_empty_q_indptr_is_refused_by_the_library(lib):
    """The shape object carries any q_indptr; what is wrong with it the library says."""
    s = native.Shape([], 4, 8)
    assert native.sd_kv8_attn_workspace_size(s) == 0 and native.sd_verify_attn_workspace_size(s) == 0
    assert _attn(lib, s) == BAD


@pytest.mark.parametrize("kw", [dict(rows=FAKE + 512), dict(row_indptr=FAKE + 512), dict(new_held=FAKE + 128), dict(table=FAKE),
                                dict(new_ctx=FAKE + 256), dict(new_ctx=FAKE + 448), dict(table=FAKE + 320),
                                dict(indptr=[0, 3, 5], path=FAKE + 512, max_path=4), dict(rows=FAKE + 900, row_indptr=FAKE + 900)])
def test_pages_extend_refuses_arrays_that_are_written_twice(lib, kw):
    assert _extend(lib, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(new_count=FAKE + 192), dict(new_held=FAKE + 256), dict(free=FAKE + 320)])
def test_pages_release_refuses_arrays_that_are_written_twice(lib, kw):
    assert _release(lib, **kw) == BAD
