"""The block-scaled cache's append and attention on the GPU, through the C ABI, against the float64 oracle.

Tolerance of the attention, per output element, derived from its roundings (half steps relative to the value):
  2^-8 |ref|          the bf16 output
  2^-7 A              the softmax weights as an e4m3 value (2^-4) and an e5m2 rest (2^-3 of at most 2^-4);
                      A = sum of p |v| / sum of p bounds any convex mix
  2 ds A              an absolute error ds of the scores changes a weight by at most e^ds - 1, in sum and in share
  2^-17 max|v_new|    the draft values as two e4m3 terms: a row is scaled so that its amax is 224..448, and what the
                      two terms leave is at most half of e4m3's smallest step 2^-9, so 2^-10 / 224 of amax < 2^-17
with ds the same error of q (2^-17 amax |k|_1 scale) and of the draft keys (2^-17 amax |q|_1 scale), and 2^-20 of
the score scale |q|_1 |k|_inf for fp32 products and sums.
The log-sum-exp is off by at most ds plus fp32 rounding of sums and logarithm (2^-20 of its size).
"""
import numpy as np
import pytest
import torch

import oracle.kv8_oracle as kv8
from speculative_decoding_verify_decode_gb300 import native, synth
from speculative_decoding_verify_decode_gb300.step import Kv8Cache, Kv8Step

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def cu(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).cuda()


def np64(t):
    return t.detach().double().cpu().numpy()


def bf16(rng, *shape, size=1.0):
    return (torch.from_numpy(rng.normal(size=shape).astype(np.float32)) * size).bfloat16()


def tree(seed, budget):
    return synth.ddtree_parents(np.random.default_rng(seed), budget)[0].tolist()


def chain(n):
    return [-1] + list(range(n - 1))


class Case:
    """One layer's inputs; pages nobody holds and slots behind a context are NaN codes, their scales NaN."""

    def __init__(self, parents, ctx, heads=(24, 4, 256), seed=0, size=1.0, spread=1.0, window=0, softcap=0.0, slopes=None,
                 scale=0.0, max_pages=None):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.dim = heads
        self.window, self.softcap, self.scale = window, softcap, scale
        self.indptr = np.cumsum([0] + [len(p) for p in parents])
        self.parents, self.ctx = np.concatenate(parents).astype(np.int32), np.array(ctx, np.int32)
        counts = [-(-c // PAGE) for c in ctx]
        pool = sum(counts) + 3
        perm = rng.permutation(pool)
        self.table = np.full((len(ctx), max_pages or max(1, max(counts))), -1, np.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (pool, self.hkv, PAGE, self.dim)
        self.codes, self.scales = {}, {}
        for c in "kv":
            x = rng.normal(size=shape).astype(np.float32) * np.exp2(rng.uniform(-spread, spread, shape[:2]))[..., None, None]
            amax = np.abs(x).max(axis=(2, 3))
            s = np.exp2(np.ceil(np.log2(amax / 448)))
            t = torch.from_numpy((x * size / (s * size)[..., None, None]).astype(np.float32)).to(torch.float8_e4m3fn)
            codes, s = t.view(torch.uint8).numpy().copy(), (s * size).astype(np.float32)
            live = np.zeros((pool, PAGE), bool)
            for b, n in enumerate(ctx):
                for j in range(counts[b]):
                    live[self.table[b, j], :max(0, min(PAGE, n - j * PAGE))] = True
            codes.transpose(0, 2, 1, 3)[~live] = 0x7F
            s[~live.any(axis=1)] = np.nan
            self.codes[c], self.scales[c] = codes, s
        n = self.indptr[-1]
        self.q, self.kn, self.vn = bf16(rng, n, self.hq, self.dim, size=size), bf16(rng, n, self.hkv, self.dim, size=size), \
            bf16(rng, n, self.hkv, self.dim, size=size)
        self.slopes = None if slopes is None else np.asarray(slopes, np.float32)

    def upload(self):
        self.d = dict(q=self.q.cuda(), k_cache=cu(self.codes["k"]), v_cache=cu(self.codes["v"]), k_scales=cu(self.scales["k"]),
                      v_scales=cu(self.scales["v"]), k_new=self.kn.cuda(), v_new=self.vn.cuda(), page_table=cu(self.table),
                      ctx_lens=cu(self.ctx), parents=cu(self.parents))
        self.shape = native.Shape(self.indptr, self.table.shape[1], len(self.codes["k"]), window=self.window,
                                  num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.dim)
        self.out = torch.full((int(self.indptr[-1]) + 1, self.hq, self.dim), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((int(self.indptr[-1]), self.hq), 7.0, device="cuda")
        self.ws = torch.full((native.sd_kv8_attn_workspace_size(self.shape) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kw = dict(scale=self.scale, softcap=self.softcap, slopes=None if self.slopes is None else cu(self.slopes))
        return self

    def call(self, **kw):
        a = dict(workspace=self.ws, dev_status=self.status, lse=self.lse, **self.kw)
        a.update(kw)
        d = self.d
        native.sd_kv8_attn(self.shape, d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], d["k_new"], d["v_new"],
                           d["page_table"], d["ctx_lens"], d["parents"], self.out[:-1], **a)

    def ref(self, only=None):
        return kv8.attention(np64(self.q), self.codes["k"], self.codes["v"], self.scales["k"], self.scales["v"], np64(self.kn),
                             np64(self.vn), self.table, self.ctx, self.indptr, self.parents, scale=self.scale or None,
                             softcap=self.softcap, slopes=self.slopes, window=self.window, only=only)

    def score_error(self):
        k1 = kinf = 0.0
        for b, n in enumerate(self.ctx):
            pages = self.table[b, :-(-int(n) // PAGE)]
            if len(pages):
                k = np.abs(kv8.dequantise(self.codes["k"][pages], self.scales["k"][pages]))
                k1, kinf = max(k1, np.nanmax(k.sum(-1))), max(kinf, np.nanmax(k))
        kn, q = np.abs(np64(self.kn)), np.abs(np64(self.q))
        k1, kinf = max(k1, kn.sum(-1).max()), max(kinf, kn.max())
        scale = self.scale or self.dim ** -0.5
        bias = 0.0 if self.slopes is None else 2.0 ** -23 * float(np.abs(self.slopes).max()) * (float(self.ctx.max()) + 64)
        q1 = q.sum(-1).max()
        return (2.0 ** -17 * (q.max() * k1 + kn.max() * q1) + 2.0 ** -20 * q1 * kinf) * scale + bias

    def check(self, only=None):
        torch.cuda.synchronize()
        assert int(self.status) == 0
        ref, lse, spread = self.ref(only)
        at = ~np.isnan(lse)
        got, got_lse, ds = np64(self.out[:-1]), np64(self.lse), self.score_error()
        assert ds < 0.25, ds
        bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2 * np.expm1(ds)) * spread + \
            2.0 ** -17 * float(self.vn.abs().max()) + 1e-30
        over = (np.abs(got - ref) / bound)[at]
        assert np.isfinite(got[at]).all() and over.max() <= 1.0, (over.max(), ds)
        assert np.all(np.abs(got_lse - lse)[at] <= ds + 2.0 ** -20 * (np.abs(lse[at]) + 1)), np.abs(got_lse - lse)[at].max()
        assert torch.all(self.out[-1] == 7.0), "rows behind the last are left as they were"
        return float(over.max())


NARROW = (32, 8, 128)
CASES = {
    "decode_one_key": ([chain(1)], [0]),
    "decode_ctx1": ([chain(1)], [1]),
    "decode_ctx15": ([chain(1)], [15]),
    "decode_ctx16": ([chain(1)], [16]),
    "decode_ctx17": ([chain(1)], [17]),
    "decode_ctx127": ([chain(1)], [127]),
    "decode_ctx128": ([chain(1)], [128]),
    "decode_ctx129_narrow": ([chain(1)], [129], NARROW),
    "chain5_ctx1000": ([chain(5)], [1000]),
    "tree23_ctx3000": ([tree(1, 22)], [3000]),
    "tree24_ctx777": ([tree(2, 23)], [777]),
    "tree25_ctx515": ([tree(3, 24)], [515]),
    "tree64_ctx300": ([tree(4, 63)], [300]),
    "tree64_narrow_ctx4100": ([tree(4, 63)], [4100], NARROW),
    "empty_context_tree": ([tree(6, 22)], [0]),
    "ragged": ([chain(1), chain(5), tree(3, 22), chain(9), tree(4, 63)], [0, 1, 17, 700, 2049]),
    "ragged_narrow": ([chain(2), tree(5, 30), chain(1), chain(3)], [33, 1500, 0, 640], NARROW),
    "decode_batch": ([chain(1)] * 40, [(37 * i * i) % 700 for i in range(40)], NARROW),
    "decode_batch_wide": ([chain(1)] * 64, [(53 * i) % 900 for i in range(64)]),
    "chain5_batch_wide": ([chain(5)] * 40, [(71 * i) % 1300 for i in range(40)]),
    "chain8_batch_narrow": ([chain(8)] * 50, [(67 * i) % 1100 for i in range(50)], NARROW),
    "batch_of_32": ([chain(1 + i % 3) for i in range(32)], [(83 * i) % 500 for i in range(32)], NARROW),
    "batch_of_33": ([chain(1 + i % 3) for i in range(33)], [(83 * i) % 500 for i in range(33)], NARROW),
    "batch_of_256": ([chain(1)] * 256, [(29 * i) % 300 for i in range(256)], (4, 2, 128)),
    "tree15_batch": ([tree(5, 14)] * 40, [(59 * i) % 700 for i in range(40)]),
    "group1": ([tree(7, 11)], [401], (3, 3, 128)),
    "group16": ([tree(8, 6), chain(1)], [401, 90], (16, 1, 256)),
    "group5_narrow": ([tree(9, 20)], [1111], (10, 2, 128)),
    "group9_wide_nodes": ([tree(9, 63)], [200], (9, 1, 256)),
    "many_heads": ([chain(3)], [260], (64, 64, 128)),
    "long_32k": ([chain(2)], [32771], (8, 1, 256)),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_attention_matches_oracle(name):
    c = Case(*CASES[name], seed=len(name)).upload()
    c.call()
    c.check()


MODS = {
    "window1": dict(window=1), "window7": dict(window=7), "window100": dict(window=100), "window129": dict(window=129),
    "window700": dict(window=700), "window5000": dict(window=5000), "window_largest": dict(window=2 ** 31 - 1), "softcap": dict(softcap=30.0),
    "tight_softcap": dict(softcap=0.5), "bias": dict(slopes=True), "bias_and_cap": dict(softcap=5.0, slopes=True),
    "all": dict(softcap=5.0, slopes=True, window=333), "scale": dict(scale=0.3),
}


@pytest.mark.parametrize("heads", [(24, 4, 256), (12, 4, 128)], ids=["d256", "d128"])
@pytest.mark.parametrize("name", sorted(MODS))
def test_score_options(name, heads):
    kw = dict(MODS[name])
    if kw.get("slopes"):
        kw["slopes"] = 2.0 ** (-8.0 * np.arange(1, heads[0] + 1) / heads[0])
    c = Case([tree(11, 17), chain(9), chain(1)], [1300, 90, 641], heads, seed=5, **kw).upload()
    c.call()
    c.check()


@pytest.mark.parametrize("seed,size,spread", [(1, 2.0, 1.0), (2, 1.0, 5.0), (3, 0.01, 2.0), (4, 3.0, 0.0)])
def test_peaked_flat_and_uneven_blocks(seed, size, spread):
    """Scores from nearly equal to one key taking all; block scales that differ by up to 2^10."""
    c = Case([tree(seed, 22), chain(4)], [2500, 700], seed=seed, size=size, spread=spread).upload()
    if spread == 5.0:
        c.q = c.q / 16
        c.upload()
    c.call()
    c.check()


def test_rising_scores_raise_the_maximum_again_and_again():
    """Each tile's scores lie far above the last one's, beyond what fp32 exponentials of an old maximum can hold."""
    c = Case([tree(2, 12)], [1500], seed=3)
    c.q[:] = 1.0
    c.codes["k"][:] = np.where(c.codes["k"] == 0x7F, 0x7F, 0x38)          # 1.0 each
    for j, page in enumerate(c.table[0]):
        c.scales["k"][page] = 2.0 ** -4 * (j // 3 + 1)                     # score 16 * scale: up to 32 in steps of 1
    c.upload()
    c.call()
    c.check()
    for j, page in enumerate(c.table[0]):
        c.scales["k"][page] = 2.0 ** -2 * (j // 2 + 1)                     # up to 188
    c.upload()
    c.call()
    c.check()


def test_flat_background_below_a_peak():
    """One key far above thousands of equal ones: the small weights still add up."""
    for gap in (6.0, 11.0, 15.0):
        c = Case([chain(2)], [6000], (4, 1, 256), seed=4)
        c.q[:] = 0.5
        c.codes["k"][:] = np.where(c.codes["k"] == 0x7F, 0x7F, 0x08)      # 2^-6 each
        c.scales["k"][c.table[0]] = 1.0
        c.kn[:] = 2.0 ** -6
        c.codes["k"][c.table[0, 3], 0, 5] = 0x38
        c.scales["k"][c.table[0, 3]] = gap / 8 + 2.0 ** -6                 # the page's other keys move little
        c.codes["v"][:] = np.where(c.codes["v"] == 0x7F, 0x7F, 0x38)
        c.codes["v"][c.table[0, 3], 0, 5] = 0xB8
        c.scales["v"][c.table[0]] = 1.0
        c.vn[:] = 1.0
        c.upload()
        c.call()
        c.check()


def test_flat_background_behind_a_peak_in_long_pieces():
    """Sixty-four sequences on one context, some 200 tiles a CTA, their own token 14 nats above 16384 equal ones:
    the background is 0.0136 of the peak, and an output without it is off by more than the bound of 2^-7 + 2^-8."""
    c = Case([chain(1)], [16384], (8, 8, 128), seed=4)
    c.codes["k"][:] = 0x08                                            # 2^-6 each
    c.codes["v"][:], c.scales["v"][:] = 0x78, 2.0 ** -8               # 1 each, as an append scales it (and the peak)
    c.scales["k"][:] = 1.0
    c.q[:], c.kn[:], c.vn[:] = 0.5, 14.0 / (0.5 * 128 ** 0.5) + 2.0 ** -6, -1.0
    ds = c.score_error()                                              # the same for every sequence
    c.score_error = lambda: ds
    c.q, c.kn, c.vn = (x.expand(64, -1, -1).contiguous() for x in (c.q, c.kn, c.vn))
    c.indptr, c.parents = np.arange(65), np.full(64, -1, np.int32)
    c.ctx, c.table = np.full(64, 16384, np.int32), np.tile(c.table, (64, 1))
    c.upload()
    c.call()
    c.check(only={(r, h) for r in (0, 17, 63) for h in (0, 5)})


def test_block_scales_at_their_ends():
    """All-zero V blocks with the smallest scale, tiny and huge scales beside ordinary ones."""
    c = Case([tree(5, 9)], [700], seed=6)
    for j in (0, 5, 6, 20):
        c.codes["v"][c.table[0, j]] = 0
        c.scales["v"][c.table[0, j]] = 2.0 ** -100
    for j in (1, 9):
        c.codes["k"][c.table[0, j]] = 0
        c.scales["k"][c.table[0, j]] = 2.0 ** -100
    c.scales["v"][c.table[0, 11]] *= 2.0 ** -60
    c.upload()
    c.call()
    c.check()
    c.codes["v"][c.table[0, :43]] = 0                                       # every full block: only the rest counts
    c.scales["v"][c.table[0, :43]] = 2.0 ** -100
    c.upload()
    c.call()
    c.check()


def test_every_finite_code():
    finite = np.array([x for x in range(256) if x & 0x7F != 0x7F], np.uint8)
    c = Case([tree(8, 22), chain(8)], [700, 333], seed=8)
    for i, x in enumerate("kv"):
        c.codes[x][:] = np.resize(np.roll(finite, 37 * i), c.codes[x].shape)
        c.scales[x][:] = 2.0 ** -9
    c.upload()
    c.call()
    c.check()


def test_masked_places_may_hold_anything():
    """NaN and infinities on other branches, behind the context and before the window reach nobody who does not see them."""
    par = [-1, 0, 0, 1, 2, 2]
    c = Case([par], [200], seed=9)
    clean = Case([par], [200], seed=9).upload()
    clean.call()
    c.kn[1], c.vn[1], c.kn[4, 2], c.vn[5, 1, 7] = float("nan"), float("inf"), float("inf"), float("nan")
    c.q[3] = float("nan")
    c.upload()
    c.call()
    torch.cuda.synchronize()
    got, want = np64(c.out[:-1]), np64(clean.out[:-1])
    for row in (0, 2):
        np.testing.assert_array_equal(got[row], want[row])
    assert np.isnan(got[3]).all() and np.isnan(got[1]).all()
    group = 6
    assert np.isnan(got[4, 2 * group:3 * group]).all() and np.isfinite(got[4, :2 * group]).all()
    np.testing.assert_array_equal(got[4, 3 * group:], want[4, 3 * group:])
    assert np.isnan(got[5, group:2 * group]).any() and np.isfinite(got[5, :group]).all()
    # a window: positions before every node's window, and one that only the shallower nodes see
    c = Case([chain(4)], [500], seed=10, window=100)
    clean = Case([chain(4)], [500], seed=10, window=100).upload()
    clean.call()
    for pos, both in ((395, True), (400, True), (402, False)):              # 401 is the root's oldest position
        page, t = c.table[0, pos // PAGE], pos % PAGE
        c.codes["v"][page, :, t] = 0x7F
        c.codes["k"][page, :, t] = 0xFF if both else c.codes["k"][page, :, t]
    c.upload()
    c.call()
    torch.cuda.synchronize()
    got, want = np64(c.out[:-1]), np64(clean.out[:-1])
    assert np.isnan(got[:2]).any(axis=(1, 2)).all()                         # nodes 0 and 1 see 402
    np.testing.assert_array_equal(got[2:], want[2:])


def test_bad_pages_and_scales_are_reported():
    for bad in (-1, -7, 10 ** 6):
        c = Case([tree(3, 9)], [600], seed=11)
        zero = Case([tree(3, 9)], [600], seed=11)
        page = int(c.table[0, 20])
        c.table[0, 20] = bad
        zero.codes["k"][page] = zero.codes["v"][page] = 0
        c.upload()
        zero.upload()
        c.call()
        zero.call()
        torch.cuda.synchronize()
        assert int(c.status) == native.SD_DEV_BAD_PAGE
        np.testing.assert_allclose(np64(c.out), np64(zero.out), atol=0.02)
    for value in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 101):
        c = Case([chain(3)], [600], seed=11)
        c.scales["v"][c.table[0, 3]] = value
        c.upload()
        c.call()
        torch.cuda.synchronize()
        assert int(c.status) & native.SD_DEV_BAD_SCALE
    for n in (-3, 10 ** 5):
        c = Case([chain(3), chain(2)], [600, 40], seed=12)
        c.ctx[1] = n
        c.table[1] = c.table[0]
        c.upload()
        c.call()
        torch.cuda.synchronize()
        assert int(c.status) & native.SD_DEV_BAD_CTX
    c = Case([[-1, 0, 2, 1]], [100], seed=12)
    c.upload()
    c.call()
    torch.cuda.synchronize()
    assert int(c.status) == native.SD_DEV_BAD_PARENTS


def test_rows_that_lie_apart():
    """q, k and v as slices of one projection's output give the bits of dense ones."""
    c = Case([tree(3, 12), chain(2)], [300, 64], seed=13).upload()
    c.call()
    want = c.out.clone()
    n, width = c.indptr[-1], (c.hq + 2 * c.hkv)
    fused = torch.full((n, width, c.dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    parts = fused[:, :c.hq], fused[:, c.hq:c.hq + c.hkv], fused[:, c.hq + c.hkv:]
    for name, p in zip(("q", "k_new", "v_new"), parts):
        p.copy_(c.d[name])
        c.d[name] = p
    c.out.fill_(7.0)
    c.call()
    assert torch.equal(c.out, want)


def test_streams_and_graphs():
    """Two calls at once on two streams with a workspace each, and captured graphs replayed on changed inputs."""
    a = Case([tree(3, 22)], [2000], seed=14).upload()
    b = Case([chain(5)] * 3, [900, 33, 1400], seed=15).upload()
    a.call()
    b.call()
    want = a.out.clone(), b.out.clone()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for c, s in zip((a, b), streams):
            s.wait_stream(torch.cuda.current_stream())
            c.out.fill_(7.0)
            s.wait_stream(torch.cuda.current_stream())
            c.call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
            c.call()
        graphs.append(g)
    a.ctx[0] = 1777
    a.d["ctx_lens"].fill_(1777)                  # a shorter context in the same graph
    for _ in range(3):
        for c, g in zip((a, b), graphs):
            c.out.fill_(7.0)
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, want[1])
    a.check()


def test_the_same_call_gives_the_same_bits():
    c = Case([tree(3, 22), chain(9)], [5000, 777], seed=16).upload()
    c.call()
    want, lse = c.out.clone(), c.lse.clone()
    for _ in range(20):
        c.ws.random_(0, 256)
        c.call()
        assert torch.equal(c.out, want) and torch.equal(c.lse, lse)


def test_a_pool_beyond_32_bit_offsets():
    """The sequence's pages lie past 2^31 codes and past 2^32 bytes of the pool."""
    heads, pool = (8, 4, 256), 270000                       # 16 KB of codes a page
    c = Case([chain(3)], [1000], heads, seed=17).upload()
    far = torch.arange(pool - 70, pool - 70 + len(c.codes["k"]), device="cuda")
    d = c.d
    for name in ("k_cache", "v_cache"):
        big = torch.empty((pool, 4, PAGE, 256), dtype=torch.uint8, device="cuda")
        big[far] = d[name]
        d[name] = big
    for name in ("k_scales", "v_scales"):
        big = torch.ones((pool, 4), device="cuda")
        big[far] = d[name]
        d[name] = big
    d["page_table"] = torch.where(d["page_table"] >= 0, d["page_table"] + pool - 70, -1).int()
    c.shape = native.Shape(c.indptr, c.table.shape[1], pool, num_q_heads=8, num_kv_heads=4)
    c.call()
    c.check()
    # the append writes there too
    new = bf16(np.random.default_rng(1), 16, 4, 256).cuda()
    slots = torch.arange(16, dtype=torch.int32, device="cuda") + (pool - 1) * PAGE
    native.sd_kv8_append([d["k_cache"]], [d["v_cache"]], [d["k_scales"]], [d["v_scales"]], [new], [new], slots)
    want, s = kv8.append(np.zeros((1, 4, PAGE, 256), np.uint8), np.ones((1, 4)), np64(new), list(range(16)))
    np.testing.assert_array_equal(d["v_cache"][-1].cpu().numpy(), want[0])
    np.testing.assert_array_equal(np64(d["v_scales"][-1]), s[0])


@pytest.mark.parametrize("name", ["ddtree22_ctx32k", "ddtree22_ctx128k", "decode_b64"])
def test_full_size_sampled(name):
    if name == "decode_b64":
        c = Case([chain(1)] * 64, [(7919 * (i + 1)) % 8000 + 1 for i in range(64)], NARROW, seed=18).upload()
        only = {(r, h) for r in (0, 5, 40, 63) for h in (0, 13, 31)}
    else:
        c = Case([tree(18, 22)], [32768 if "32k" in name else 131072], seed=18).upload()
        only = {(r, h) for r in (0, 7, 22) for h in (0, 9, 23)}
    c.call()
    c.check(only)


# ------------------------------------------------------------------------------------------ append

def _append_check(pages, heads, dim, layers, slots, src_rows, rows=None, seed=0, special=None, old_scale=None, strided=False):
    rng = np.random.default_rng(seed)
    codes = [[rng.integers(0, 256, (pages, heads, PAGE, dim)).astype(np.uint8) for _ in range(layers)] for _ in "kv"]
    scales = [[np.exp2(rng.integers(-12, -6, (pages, heads))).astype(np.float32) for _ in range(layers)] for _ in "kv"]
    if old_scale is not None:
        for per in scales:
            for s in per:
                s[:] = old_scale
    for per in codes:
        for c in per:
            c[(c & 0x7F) == 0x7F] = 0x31
    new = [[bf16(rng, src_rows, heads, dim) * 2.0 ** float(rng.integers(-3, 4)) for _ in range(layers)] for _ in "kv"]
    if special is not None:
        special(new, codes, scales)
    dc, ds = [[cu(x) for x in per] for per in codes], [[cu(x) for x in per] for per in scales]
    dn = [[x.cuda() for x in per] for per in new]
    if strided:
        wide = [[torch.full((src_rows, heads + 3, dim), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in per] for per in dn]
        for w, x in zip(sum(wide, []), sum(dn, [])):
            w[:, 1:1 + heads] = x
        dn = [[w[:, 1:1 + heads] for w in per] for per in wide]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.sd_kv8_append(dc[0], dc[1], ds[0], ds[1], dn[0], dn[1], cu(slots, torch.int32),
                         None if rows is None else cu(rows, torch.int32), status)
    torch.cuda.synchronize()
    for per_c, per_s, per_n, gc, gs in zip(codes, scales, new, dc, ds):
        for c, s, x, g, h in zip(per_c, per_s, per_n, gc, gs):
            want, ws = kv8.append(c, s, np64(x), slots, rows)
            got = g.cpu().numpy()
            nan = (want & 0x7F) == 0x7F
            assert np.array_equal((got & 0x7F) == 0x7F, nan)
            np.testing.assert_array_equal(got[~nan], want[~nan])
            np.testing.assert_array_equal(np64(h), ws)
    return int(status)


def _slots(rng, pages, runs):
    """Slot map of sequences: (first offset, rows) each on pages of their own, with -1 behind."""
    perm, at, out = rng.permutation(pages), 0, []
    for off, n in runs:
        for i in range(n):
            out.append(int(perm[at + (off + i) // PAGE]) * PAGE + (off + i) % PAGE)
        at += (off + max(n, 1) - 1) // PAGE + 1
    assert at <= pages
    return out + [-1] * 3


@pytest.mark.parametrize("heads,dim", [(4, 256), (8, 128), (1, 128), (3, 256)])
@pytest.mark.parametrize("runs", [[(0, 1)], [(15, 1)], [(7, 3), (0, 0), (15, 2), (0, 16)], [(5, 100), (0, 33), (14, 1)],
                                  [(i % 16, 1) for i in range(40)]], ids=["one", "last", "mixed", "prompts", "decode"])
def test_append_matches_oracle(heads, dim, runs):
    slots = _slots(np.random.default_rng(1), 60, runs)
    assert _append_check(60, heads, dim, 2, slots, len(slots), seed=len(slots)) == 0


def test_append_a_long_prompt_takes_sixteen_rows_a_block():
    slots = _slots(np.random.default_rng(2), 400, [(3, 2500), (0, 1700), (15, 18)])
    assert _append_check(400, 2, 256, 1, slots, len(slots), seed=3) == 0


def test_append_source_rows_and_strides():
    slots = _slots(np.random.default_rng(3), 9, [(4, 20), (0, 5)])
    rows = list(np.random.default_rng(4).permutation(70)[:25]) + [0, -1, 999]      # behind -1 slots: not read
    assert _append_check(9, 4, 256, 3, slots, 70, rows, seed=5, strided=True) == 0


def test_append_special_values():
    def plant(new, codes, scales):
        vals = torch.tensor([448.0, 449.0, 464.0, 1e30, -1e30, float("inf"), float("-inf"), 0.0, -0.0, float("nan"),
                             2.0 ** -9, 3 * 2.0 ** -11, 1e-38])
        new[0][0][0, 0, :13] = vals.bfloat16()
        new[0][0][1, 1] = float("nan")
        new[0][0][2, 2] = 0.0
        new[1][0][3] = 3e38
        new[1][0][4:8] = 0.0
        new[1][0][8:12] = torch.tensor(1e-35).bfloat16()
    slots = [0, 17, 33, 48] + [64 + i for i in range(4)] + [80 + i for i in range(4)]
    assert _append_check(8, 4, 256, 1, slots, 12, seed=6, special=plant) == 0


@pytest.mark.parametrize("old", [2.0 ** -100, 2.0 ** -20, 0.3, 2.0 ** 100])
def test_append_behind_old_scales(old):
    """Growth from the smallest scale, a scale that is no power of two, and one that stays."""
    slots = _slots(np.random.default_rng(7), 12, [(9, 30), (1, 2), (15, 1)])
    assert _append_check(12, 4, 256, 1, slots, len(slots), seed=8, old_scale=old) == 0


def test_append_refuses_broken_maps():
    def run(slots, rows=None, src=8, pool=6):
        k = torch.full((pool, 4, PAGE, 256), 9, dtype=torch.uint8, device="cuda")
        s = torch.full((pool, 4), 0.5, device="cuda")
        x = torch.ones(src, 4, 256, dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        native.sd_kv8_append([k], [k.clone()], [s], [s.clone()], [x], [x], cu(slots, torch.int32),
                             None if rows is None else cu(rows, torch.int32), st)
        torch.cuda.synchronize()
        return int(st), k
    for slots, rows in [([96], None), ([-2], None), ([2 ** 31 - 1], None), ([3, 3], None), ([3, 5], None), ([5, 4], None),
                        ([0], [8]), ([0], [-1]), ([0, 1], [0, 2 ** 30]), ([0] * 1 + [1] * 1 + [1], None)]:
        st, k = run(slots, rows)
        assert st == native.SD_DEV_BAD_SLOT and torch.all(k == 9), (slots, rows)
    st, k = run([0, 1, 96, 32])
    assert st == native.SD_DEV_BAD_SLOT and torch.all(k[2, :, 0] != 9) and torch.all(k[0, :, :2] != 9)
    assert run([i for i in range(12)], src=8)[0] == native.SD_DEV_BAD_SLOT        # more rows than sources
    assert run([], None)[0] == 0 and run([-1, -1])[0] == 0
    for old in (0.0, float("nan"), -1.0, float("inf")):
        k = torch.full((2, 4, PAGE, 256), 9, dtype=torch.uint8, device="cuda")
        s = torch.full((2, 4), old, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        x = torch.ones(1, 4, 256, dtype=torch.bfloat16, device="cuda")
        native.sd_kv8_append([k], [k.clone()], [s], [s.clone()], [x], [x], cu([5], torch.int32), None, st)
        assert int(st) == native.SD_DEV_BAD_SCALE and torch.all(k == 9)
        st.zero_()
        native.sd_kv8_append([k], [k.clone()], [s], [s.clone()], [x], [x], cu([16], torch.int32), None, st)   # begins a page
        assert int(st) == 0 and torch.all(s[1] == 2.0 ** -8)


# ------------------------------------------------------------------------------------------ the operators together

@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_prompt_then_verify_steps(graph):
    """Prompts join, then verify steps run over the growing cache; every step's attention, tokens, pages and codes
    follow the oracle's, and the pages return at the end."""
    layers, heads, dim, hq, vocab = 2, 4, 256, 24, 97
    par = [tree(1, 10), chain(4), chain(1)]
    indptr = np.cumsum([0] + [len(p) for p in par])
    parents, total = np.concatenate(par).astype(np.int32), int(indptr[-1])
    cache = Kv8Cache(3, 40, 64, layers)
    step = Kv8Step(cache, indptr, vocab, softcap=20.0)
    rng = np.random.default_rng(3)
    lens = [200, 31, 0]
    prompt = [[bf16(rng, 240, heads, dim) for _ in range(layers)] for _ in "kv"]
    slots = torch.empty(240, dtype=torch.int32, device="cuda")
    cache.extend(cu(lens, torch.int32), [x.cuda() for x in prompt[0]], [x.cuda() for x in prompt[1]], slots)
    codes = [[np.zeros((64, heads, PAGE, dim), np.uint8) for _ in range(layers)] for _ in "kv"]
    scales = [[np.ones((64, heads)) for _ in range(layers)] for _ in "kv"]
    table, held, free = np.full((3, 40), -1), [0, 0, 0], list(range(63, -1, -1))
    table, held, free, sl, _, _, ctx = kv8.pages_extend([0, 0, 0], lens, table, held, free, 240)
    put = lambda new, sl, rows: [[kv8.append(c, s, np64(x), sl, rows) for c, s, x in zip(a, b, n)] for a, b, n in zip(codes, scales, new)]
    done = put(prompt, sl, None)
    buf = dict(q=torch.empty(layers, total, hq, dim, dtype=torch.bfloat16, device="cuda"),
               k=torch.empty(layers, total, heads, dim, dtype=torch.bfloat16, device="cuda"),
               v=torch.empty(layers, total, heads, dim, dtype=torch.bfloat16, device="cuda"),
               logits=torch.empty(total, vocab, device="cuda"), draft=torch.zeros(total, dtype=torch.int32, device="cuda"))
    run = lambda: step.run(buf["q"], buf["k"], buf["v"], cu(parents) if not graph else dpar, buf["draft"], buf["logits"])
    dpar = cu(parents)
    g = None
    for it in range(4):
        codes = [[c for c, _ in per] for per in done]
        scales = [[s for _, s in per] for per in done]
        q, kn, vn = bf16(rng, layers, total, hq, dim), bf16(rng, layers, total, heads, dim, size=2.0 ** it), bf16(rng, layers, total, heads, dim)
        logits = rng.normal(size=(total, vocab)).astype(np.float32)
        t = logits.argmax(1)
        draft = np.array([0 if parents[r] < 0 else (t[indptr[b] + parents[r]] if rng.random() < 0.8 else 1 + t[r] % 5)
                          for b in range(3) for r in range(indptr[b], indptr[b + 1])], np.int32)
        for name, x in (("q", q), ("k", kn), ("v", vn)):
            buf[name].copy_(x)
        buf["logits"].copy_(torch.from_numpy(logits))
        buf["draft"].copy_(torch.from_numpy(draft))
        if graph and g is None:
            state = [x.clone() for x in (cache.ctx_lens, cache.held, cache.free_count)]
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run()
            for x, y in zip((cache.ctx_lens, cache.held, cache.free_count), state):
                assert torch.equal(x, y)                      # a capture runs nothing
        g.replay() if graph else run()
        torch.cuda.synchronize()
        assert int(cache.dev_status) == 0
        import oracle
        _, alen, paths, toks = oracle.accept(indptr, parents, draft, logits)
        assert list(step.accept_len.cpu().numpy()) == list(alen)
        for layer in range(layers):
            ref, _, spread = kv8.attention(np64(q[layer]), codes[0][layer], codes[1][layer], scales[0][layer], scales[1][layer],
                                           np64(kn[layer]), np64(vn[layer]), table, ctx, indptr, parents, softcap=20.0)
            got = np64(step.out[layer])
            ds = 2.0 ** -16 * float(q.abs().max()) * 256 * 4 * 2.0 ** it / 16       # |k|_1 <= 256 values of up to 4 * 2^it
            assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2 * np.expm1(ds)) * spread +
                          2.0 ** -17 * float(vn.abs().max()))
        table, held, free, sl, rows, _, ctx = kv8.pages_extend(ctx, alen, table, held, free, total, indptr, paths)
        assert list(step.slots.cpu().numpy()) == sl and list(step.rows.cpu().numpy()) == rows
        done = put([list(kn), list(vn)], sl, rows)
        for per, gc, gs in zip(done, (cache.k, cache.v), (cache.k_scales, cache.v_scales)):
            for layer, (c, s) in enumerate(per):
                np.testing.assert_array_equal(gc[layer].cpu().numpy(), c)
                np.testing.assert_array_equal(np64(gs[layer]), s)
        assert list(cache.ctx_lens.cpu().numpy()) == ctx and list(cache.held.cpu().numpy()) == held
        assert int(cache.free_count) == len(free)
    cache.release(cu([100, 0, 10 ** 6], torch.int32))
    held, free = kv8.pages_release([100, 0, 10 ** 6], table, held, free)
    assert list(cache.held.cpu().numpy()) == held and int(cache.free_count) == len(free)
    assert list(cache.free_list.cpu().numpy()[:len(free)]) == free
    assert list(cache.ctx_lens.cpu().numpy()) == [100, 0, ctx[2]]


@pytest.mark.parametrize("raw", [False, True], ids=["torch_stream", "handle"])
def test_a_refused_release_leaves_the_cache_as_it_was(raw):
    cache, rng = Kv8Cache(2, 8, 16, 1), np.random.default_rng(5)
    x = bf16(rng, 70, 4, 256).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stream = side.cuda_stream if raw else side
    slots = torch.empty(70, dtype=torch.int32, device="cuda")
    cache.extend(cu([50, 20], torch.int32), [x], [x], slots, stream=stream)
    side.synchronize()
    assert cache.ctx_lens.tolist() == [50, 20] and cache.held.tolist() == [4, 2] and int(cache.dev_status) == 0
    cache.release(cu([10, -1], torch.int32), stream=stream)
    side.synchronize()
    assert int(cache.dev_status) == native.SD_DEV_BAD_CTX
    assert cache.ctx_lens.tolist() == [50, 20] and cache.held.tolist() == [4, 2] and int(cache.free_count) == 10
    cache.release(cu([10, 100], torch.int32), stream=0 if raw else None)
    torch.cuda.synchronize()
    assert cache.ctx_lens.tolist() == [10, 20] and cache.held.tolist() == [1, 2] and int(cache.free_count) == 13


@pytest.mark.parametrize("heads,nodes", [((24, 4, 256), 1), ((24, 4, 256), 5), ((24, 4, 256), 13), ((24, 4, 256), 23),
                                         ((16, 16, 128), 9), ((32, 8, 128), 8), ((32, 8, 128), 31)])
def test_batches_without_context(heads, nodes):
    """Hundreds of sequences of nothing but a draft block: every CTA works through several pieces that no cache tile
    separates, with every width of its rings."""
    batch = 256 if nodes < 20 else 128
    c = Case([tree(i, nodes - 1) if nodes > 2 else chain(nodes) for i in range(batch)], [0] * batch, heads, seed=nodes).upload()
    rng, total = np.random.default_rng(nodes), int(c.indptr[-1])
    c.call()
    c.check(only={(int(rng.integers(total)), int(rng.integers(c.hq))) for _ in range(200)})
    want, lse = c.out.clone(), c.lse.clone()
    for _ in range(10):
        c.out.fill_(7.0)
        c.call()
        assert torch.equal(c.out, want) and torch.equal(c.lse, lse)
    assert int(c.status) == 0


@pytest.mark.parametrize("heads,mods", [((24, 4, 256), {}), ((32, 8, 128), {}), ((12, 4, 128), dict(softcap=30.0, slopes=True)),
                                        ((24, 4, 256), dict(slopes=True))], ids=["d256", "d128", "capped_bias", "bias"])
@pytest.mark.parametrize("power", [-20, 12, 20, 100])
def test_large_queries_leave_the_others_alone(heads, mods, power):
    """One node and one head of every group 2^12 to 2^100 times the rest (or the rest that much larger than them):
    every ordinary row keeps the bound of its own query, whose error is 2^-17 of its own amax."""
    mods = dict(mods)
    if mods.get("slopes"):
        mods["slopes"] = 2.0 ** (-8.0 * np.arange(1, heads[0] + 1) / heads[0])
    c = Case([tree(3, 12), chain(6)], [700, 90], heads, seed=19, **mods)
    group = heads[0] // heads[1]
    apart = np.zeros((int(c.indptr[-1]), heads[0]), bool)
    apart[[2, 14]] = True
    apart[:, 1::group] = True
    c.q[torch.from_numpy(apart)] *= 2.0 ** power
    c.upload()
    c.call()
    torch.cuda.synchronize()
    assert int(c.status) == 0
    ref, lse, spread = c.ref()
    got, got_lse = np64(c.out[:-1]), np64(c.lse)
    k1 = kinf = 0.0
    for b, n in enumerate(c.ctx):
        k = np.abs(kv8.dequantise(c.codes["k"][c.table[b, :-(-int(n) // PAGE)]], c.scales["k"][c.table[b, :-(-int(n) // PAGE)]]))
        k1, kinf = max(k1, np.nanmax(k.sum(-1))), max(kinf, np.nanmax(k))
    kn, q = np.abs(np64(c.kn)), np.abs(np64(c.q))
    k1, kinf = max(k1, kn.sum(-1).max()), max(kinf, kn.max())
    bias = 0.0 if c.slopes is None else 2.0 ** -23 * float(np.abs(c.slopes).max()) * (float(c.ctx.max()) + 64)
    ds = (2.0 ** -17 * (q.max(-1) * k1 + kn.max() * q.sum(-1)) + 2.0 ** -20 * q.sum(-1) * kinf) * c.dim ** -0.5 + bias   # a row's
    small = ds < 0.25
    assert np.array_equal(small, ~apart) if power > 0 else small.all()
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2 * np.expm1(np.where(small, ds, 0))[..., None]) * spread + \
        2.0 ** -17 * float(c.vn.abs().max())
    over = (np.abs(got - ref) / bound)[small]
    assert over.max() <= 1.0, over.max()
    assert np.all(np.abs(got_lse - lse)[small] <= (ds + 2.0 ** -20 * (np.abs(lse) + 1))[small])
    assert np.isfinite(got).all() and np.isfinite(got_lse).all()


@pytest.mark.parametrize("tiles", [63, 64, 255, 256, 1024])
def test_flat_backgrounds_at_every_depth(tiles):
    """One CTA a sequence and KV head, its own token 3 to 18 nats above tens of thousands of equal ones: weights of every
    size down to those that no longer reach the output, all alike, so that their roundings must not all go one way."""
    batch = 152
    c = Case([chain(1)], [128 * tiles], (2, 2, 128), seed=4)
    c.codes["k"][:] = 0x08                                            # 2^-6 each
    c.codes["v"][:], c.scales["v"][:] = 0x78, 2.0 ** -8               # 1 each, as an append scales it (and the peak)
    c.scales["k"][:] = 1.0
    c.q[:], c.vn[:] = 0.5, -1.0
    ds = c.score_error() + 2.0 ** -17 * 18.0 * 2                      # of the largest key: 2^-17 of q and of k in the score
    c.score_error = lambda: ds
    gap = torch.linspace(3.0, 18.0, batch)
    kn = (gap / (0.5 * 128 ** 0.5) + 2.0 ** -6)[:, None, None]
    c.q, c.vn = (x.expand(batch, -1, -1).contiguous() for x in (c.q, c.vn))
    c.kn = kn.expand(batch, 2, 128).bfloat16().contiguous()
    c.indptr, c.parents = np.arange(batch + 1), np.full(batch, -1, np.int32)
    c.ctx, c.table = np.full(batch, 128 * tiles, np.int32), np.tile(c.table, (batch, 1))
    c.upload()
    c.call()
    c.check(only={(r, r % 2) for r in range(0, batch, 2 if tiles < 200 else 7 if tiles < 1000 else 19)})


@pytest.mark.parametrize("apart", [8, 12, 15])
def test_value_scales_far_apart(apart):
    """Equal softmax weights on blocks whose V scales are 2^8 to 2^15 apart, the large ones zero in half of the dims: what
    the small blocks put there is off by 2^-7 of its size, or by a quarter where their weights are small."""
    c = Case([chain(2)], [640], (4, 1, 256), seed=21, spread=0.0)
    c.q[:] = 0.0
    small = c.table[0, ::2]
    c.scales["v"][small] *= 2.0 ** -apart
    c.vn *= 2.0 ** -apart
    large = c.table[0, 1:40:2]
    c.codes["v"][large, :, :, 128:] = 0
    c.upload()
    c.call()
    torch.cuda.synchronize()
    ref, _, spread = c.ref()
    got = np64(c.out[:-1])
    rel = np.where(np.arange(256) < 128, 2.0 ** -7, 2.0 ** -7 if apart <= 8 else 0.25)
    bound = 2.0 ** -8 * np.abs(ref) + rel * spread + 2.0 ** -17 * float(c.vn.abs().max())
    over = (np.abs(got - ref) / bound).max()
    assert int(c.status) == 0 and over <= 1.0, over


@pytest.mark.parametrize("heads", [(24, 4, 256), (12, 4, 128)], ids=["d256", "d128"])
@pytest.mark.parametrize("cap", [1e-38, 1e-3, 64.0, 1e3, 4096.0])
def test_every_size_of_score_cap(heads, cap):
    """A cap far above every score changes nothing, a tiny one makes all scores alike: within the bound of any call."""
    slopes = 2.0 ** (-8.0 * np.arange(1, heads[0] + 1) / heads[0]) if cap == 1e3 else None
    c = Case([tree(11, 17), chain(9), chain(1)], [1300, 90, 641], heads, seed=5, softcap=cap, slopes=slopes).upload()
    c.call()
    c.check()


@pytest.mark.parametrize("cap", [40.0, 1000.0])
def test_scores_that_reach_the_cap(cap):
    """Scores from far below to the cap itself."""
    c = Case([tree(2, 12)], [1500], seed=3, softcap=cap)
    c.q[:] = 1.0
    c.codes["k"][:] = np.where(c.codes["k"] == 0x7F, 0x7F, 0x38)          # 1.0 each: a score of 16 times the scale
    for j, page in enumerate(c.table[0]):
        c.scales["k"][page] = cap / 16 * (j + 1) / 47
    c.upload()
    c.call()
    c.check()


def test_a_release_refused_for_any_reason_leaves_the_cache_as_it_was():
    """Negative lengths, a held count out of range, a free list without room; a page id out of range is pushed all the same."""
    def cache():
        c = Kv8Cache(2, 8, 16, 1)
        x = bf16(np.random.default_rng(6), 70, 4, 256).cuda()
        c.extend(cu([50, 20], torch.int32), [x], [x], torch.empty(70, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert c.ctx_lens.tolist() == [50, 20] and c.held.tolist() == [4, 2] and int(c.free_count) == 10
        return c
    def negative(c): c.keep = [10, -1]
    def held(c): c.held[1] = 9
    def below(c): c.held[1] = -1
    def room(c): c.free_count.fill_(16)
    def count(c): c.free_count.fill_(-1)
    for plant, bit in [(negative, native.SD_DEV_BAD_CTX), (held, native.SD_DEV_BAD_CTX), (below, native.SD_DEV_BAD_CTX),
                       (room, native.SD_DEV_BAD_PAGE), (count, native.SD_DEV_BAD_PAGE)]:
        c = cache()
        c.keep = [10, 100]
        plant(c)
        state = [x.clone() for x in (c.ctx_lens, c.held, c.free_count, c.free_list, c.page_table)]
        c.release(cu(c.keep, torch.int32))
        torch.cuda.synchronize()
        assert int(c.dev_status) == bit, plant
        for x, y in zip((c.ctx_lens, c.held, c.free_count, c.free_list, c.page_table), state):
            assert torch.equal(x, y), plant
    c = cache()
    c.page_table[0, 2] = 10 ** 6
    c.release(cu([10, 18], torch.int32))
    torch.cuda.synchronize()
    assert int(c.dev_status) == native.SD_DEV_BAD_PAGE
    assert c.ctx_lens.tolist() == [10, 18] and c.held.tolist() == [1, 2] and int(c.free_count) == 13
    c.release(cu([10, 17], torch.int32))                    # no page moves, and the old status does not stand in the way
    assert c.ctx_lens.tolist() == [10, 17] and int(c.dev_status) == native.SD_DEV_BAD_PAGE
    c.release(cu([0, 0], torch.int32))
    assert c.ctx_lens.tolist() == [0, 0] and int(c.free_count) == 16


@pytest.mark.parametrize("extra", [[3], [15], [0, 1, 2]])
@pytest.mark.parametrize("rows", [20, 900])
def test_append_reports_rows_behind_a_full_page(rows, extra):
    """Sixteen rows fill a page; more on the same page break the order, and are not dropped in silence."""
    slots = list(range(32, 48)) + [32 + i for i in extra] + [64]
    slots += [-1] * (rows - len(slots))
    k = torch.full((6, 4, PAGE, 256), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((6, 4), 0.5, device="cuda")
    x = torch.ones(rows, 4, 256, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.sd_kv8_append([k], [k.clone()], [s], [s.clone()], [x], [x], cu(slots, torch.int32), None, st)
    torch.cuda.synchronize()
    assert int(st) == native.SD_DEV_BAD_SLOT and torch.all(k[2] == 9) and torch.all(k[4, :, 0] != 9)
