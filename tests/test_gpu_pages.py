"""Page tables and slot maps built on the GPU, against a plain free-list stack.  Whole numbers: equal."""
import numpy as np
import pytest
import torch

import oracle.kv8_oracle as kv8
from speculative_decoding_verify_decode_gb300 import native

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def cu(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


class Pages:
    def __init__(self, ctx, spare=5, max_pages=64, extra_held=0, seed=0):
        rng = np.random.default_rng(seed)
        held = [-(-c // 16) + extra_held for c in ctx]
        self.pool = sum(held) + spare
        perm = rng.permutation(self.pool)
        self.table, at = np.full((len(ctx), max_pages), -1), 0
        for b, n in enumerate(held):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.ctx, self.held, self.free = list(ctx), held, [int(x) for x in perm[at:]]

    def extend(self, add, max_rows, q_indptr=None, path=None, rows=True, odd=0):
        B = len(self.ctx)
        dev = lambda n, v=-9: torch.full((n,), v, dtype=torch.int32, device="cuda")
        table, free = cu(self.table), cu(self.free + [-5] * (self.pool - len(self.free)))
        o = dict(held=dev(B), count=dev(1), slots=dev(max_rows + odd + 1)[odd:odd + max_rows], rows=dev(max_rows + odd)[odd:],
                 indptr=dev(B + 1), ctx=dev(B), status=dev(1, 0))
        native.sd_pages_extend(cu(self.ctx), cu(add), table, cu(self.held), o["held"], free, cu([len(self.free)]), o["count"],
                               o["slots"], rows=o["rows"] if rows else None, row_indptr=o["indptr"], new_ctx_lens=o["ctx"],
                               q_indptr=q_indptr, path=None if path is None else cu(path), dev_status=o["status"])
        torch.cuda.synchronize()
        assert torch.equal(free, cu(self.free + [-5] * (self.pool - len(self.free))))
        return dict({k: v.cpu().tolist() for k, v in o.items()}, table=table.cpu().numpy())

    def check(self, add, max_rows, **kw):
        got = self.extend(add, max_rows, **kw)
        assert got["status"] == [0]
        path = kw.get("path")
        table, held, free, slots, rows, indptr, ctx = kv8.pages_extend(self.ctx, add, self.table, self.held, self.free, max_rows,
                                                                       kw.get("q_indptr"), path)
        assert got["held"] == held and got["count"] == [len(free)] and got["indptr"] == indptr and got["ctx"] == ctx
        assert np.array_equal(got["table"], table) and got["slots"] == slots
        assert got["rows"] == (rows if kw.get("rows", True) else [-9] * max_rows)

    def unchanged(self, add, max_rows, bits, **kw):
        got = self.extend(add, max_rows, **kw)
        assert got["status"][0] & bits == bits, got["status"]
        assert got["held"] == self.held and got["count"] == [len(self.free)] and got["ctx"] == self.ctx
        assert np.array_equal(got["table"], self.table) and got["slots"] == [-1] * max_rows == got["rows"]
        assert got["indptr"] == [0] * (len(self.ctx) + 1)


@pytest.mark.parametrize("ctx,add,extra", [([0], [1], 0), ([0], [0], 0), ([15], [1], 0), ([16], [1], 0), ([16], [17], 3),
                                           ([5, 0, 33, 16, 100], [3, 0, 31, 1, 77], 0), ([5, 0, 33], [300, 16, 1], 1),
                                           ([0] * 256, list(range(256)), 0), ([i % 40 for i in range(255)], [1] * 255, 0)])
@pytest.mark.parametrize("odd", [0, 1])
def test_extend(ctx, add, extra, odd):
    p = Pages(ctx, spare=sum(add) // 16 + len(ctx) + 1, extra_held=extra)
    p.check(add, sum(add) + odd, odd=odd)
    p.check(add, sum(add) + 37, rows=False, odd=odd)


def test_extend_takes_the_last_free_page():
    p = Pages([16, 0], spare=3)
    p.check([16, 32], 48)
    p.unchanged([17, 32], 60, native.SD_DEV_NO_PAGES)


def test_extend_long_prompts():
    rng = np.random.default_rng(1)
    ctx, add = rng.integers(0, 500, 64).tolist(), rng.integers(0, 4000, 64).tolist()
    add[3] = add[40] = 0
    p = Pages(ctx, spare=sum(add) // 16 + 64, max_pages=300)
    p.check(add, sum(add) + 11)


def test_extend_accepted_paths():
    ctx, lens = [5, 16, 0, 31], [3, 0, 1, 4]
    indptr = [0, 9, 10, 33, 40]
    path = np.full((4, 6), -1)
    path[0, :3], path[2, :1], path[3, :4] = [0, 2, 7], [0], [0, 1, 5, 6]
    p = Pages(ctx, spare=9)
    p.check(lens, 12, q_indptr=indptr, path=path)
    rng = np.random.default_rng(2)
    ctx, lens = rng.integers(0, 900, 256).tolist(), rng.integers(0, 17, 256).tolist()
    path = np.sort(rng.random((256, 20)).argsort(1)[:, :16], 1)
    Pages(ctx, spare=256).check(lens, 256 * 16, q_indptr=list(range(0, 257 * 20, 20)), path=path)


def test_extend_refuses_on_the_device():
    p = Pages([5, 20], spare=9, max_pages=4)
    for add, rows, bits in [([-1, 3], 9, native.SD_DEV_BAD_CTX), ([60, 3], 99, native.SD_DEV_BAD_CTX),
                            ([2 ** 31 - 1, 0], 9, native.SD_DEV_BAD_CTX), ([4, 5], 8, native.SD_DEV_BAD_SLOT)]:
        p.unchanged(add, rows, bits)
    p.ctx[0] = -4
    p.unchanged([1, 1], 9, native.SD_DEV_BAD_CTX)
    p.ctx[0] = 17                                           # more than its one page holds
    p.unchanged([1, 1], 9, native.SD_DEV_BAD_CTX)
    p = Pages([5, 20], spare=9)
    for held in ([-1, 2], [1, 65]):
        p.held = held
        p.unchanged([1, 1], 9, native.SD_DEV_BAD_CTX)
    p = Pages([5, 20], spare=9)
    ind, path = [0, 4, 9], np.array([[0, 1, 3], [0, 4, 2]])
    p.check([3, 2], 6, q_indptr=ind, path=path)
    for a, bad in [([3, 2], [[0, 1, 4], [0, 4, 2]]), ([3, 2], [[0, -1, 3], [0, 4, 2]]), ([4, 2], path), ([0, 6], path)]:
        p.unchanged(a, 9, native.SD_DEV_BAD_ACCEPT, q_indptr=ind, path=bad)


def test_extend_reports_pages_out_of_range():
    p = Pages([20], spare=4)
    p.free[-1] = 10 ** 6                                    # taken first
    got = p.extend([30], 30)
    assert got["status"] == [native.SD_DEV_BAD_PAGE]
    want = kv8.pages_extend(p.ctx, [30], p.table, p.held, p.free, 30)[3]
    assert got["slots"] == [-1 if s >= p.pool * 16 else s for s in want] and -1 in got["slots"]
    p = Pages([20], spare=4)
    p.table[0, 1] = -3
    got = p.extend([30], 30)
    assert got["status"] == [native.SD_DEV_BAD_PAGE] and got["slots"][:12] == [-1] * 12 and got["slots"][12] >= 0


def _release(p, keep, free=None, count=None):
    B = len(p.held)
    dev = lambda n, v=-9: torch.full((n,), v, dtype=torch.int32, device="cuda")
    lst = cu(p.free + [-5] * (p.pool - len(p.free)) if free is None else free)
    held, cnt, st = dev(B), dev(1), dev(1, 0)
    native.sd_pages_release(cu(keep), cu(p.table), cu(p.held), held, lst, cu([len(p.free) if count is None else count]), cnt, st)
    torch.cuda.synchronize()
    return held.tolist(), lst.tolist(), cnt.item(), st.item()


@pytest.mark.parametrize("ctx,keep", [([0], [0]), ([1], [0]), ([17], [16]), ([17], [17]), ([17], [10 ** 9]),
                                      ([100, 5, 0, 64], [33, 0, 9, 64]), ([i * 3 for i in range(256)], [i for i in range(256)])])
def test_release(ctx, keep):
    p = Pages(ctx, spare=4)
    held, lst, n, st = _release(p, keep)
    want_held, free = kv8.pages_release(keep, p.table, p.held, p.free)
    assert st == 0 and held == want_held and n == len(free) and lst[:n] == free and all(x == -5 for x in lst[n:])


def test_release_refuses_on_the_device():
    p = Pages([100, 50], spare=4)
    before = p.free + [-5] * (p.pool - len(p.free))
    held, lst, n, st = _release(p, [-1, 0])
    assert st == native.SD_DEV_BAD_CTX and held == p.held and lst == before and n == len(p.free)
    held, lst, n, st = _release(p, [0, 0], count=p.pool - 3)          # more pages than the list has room for
    assert st == native.SD_DEV_BAD_PAGE and held == p.held and lst == before and n == p.pool - 3
    p.table[0, 2] = 10 ** 6
    held, lst, n, st = _release(p, [0, 50])
    assert st == native.SD_DEV_BAD_PAGE and held == [0, 4] and n == len(p.free) + 7 and 10 ** 6 in lst
