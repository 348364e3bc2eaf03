"""The 4-bit cache's append, read and attention on the GPU, through the C ABI, against the float64 oracle.

Append and read are compared bit for bit.  Tolerance of the attention, per output element, derived from its roundings
(half steps relative to the value):
  2^-8 |ref|          the bf16 output
  2^-8 A              the softmax weights as bf16; A = sum of p |v| / sum of p bounds any convex mix
  2 ds A              an absolute error ds of the scores changes a weight by at most e^ds - 1, in sum and in share
  n 2^-27 A + 2^-18 A fp32 accumulation of n tokens, 16 a product, each step off by at most 2^-23 of what is summed up;
                      exponentials, sums of weights, the merge
with ds = 2^-20 |q|_1 |k|_inf scale for the fp32 products and sums of a score (and, with a bias, the rounding of slope times
distance, of capped scores 2^-21 of the cap).  Keys, values and queries enter exactly.  The log-sum-exp is off by at most ds plus fp32 rounding
of sums and logarithm (2^-20 of its size).
"""
import numpy as np
import pytest
import torch

import oracle.kv4_oracle as kv4
from speculative_decoding_verify_decode_gb300 import native, synth

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


def pack(codes_k, scales_k, codes_v, scales_v):
    """A cache uint8 [pages, heads, 2, 9 dim] from codes [pages, heads, 16, dim] and scales [pages, heads, 16, dim / 32]."""
    pages, heads, _, dim = codes_k.shape
    nb = dim // 32
    shift = np.array([kv4.bit(e) for e in range(8)], np.uint32)

    def words(c):
        return np.bitwise_or.reduce(c.reshape(*c.shape[:-1], -1, 8).astype(np.uint32) << shift, axis=-1)

    def bits(s):
        return (np.ascontiguousarray(s, np.float32).view(np.uint32) >> 16).astype("<u2")
    k = words(codes_k).reshape(pages, heads, PAGE, nb, 4).transpose(0, 1, 3, 2, 4)
    v = words(codes_v.transpose(0, 1, 3, 2))
    raw = lambda x, t: np.ascontiguousarray(x.astype(t)).view(np.uint8).reshape(pages, heads, -1)
    return np.stack([np.concatenate([raw(k, "<u4"), raw(bits(scales_k), "<u2")], -1),
                     np.concatenate([raw(v, "<u4"), raw(bits(scales_v.transpose(0, 1, 3, 2)), "<u2")], -1)], 2)


class Case:
    """One layer's inputs; pages nobody holds and slots behind a context hold NaN scales."""

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
        self.live = np.zeros((pool, PAGE), bool)
        for b, n in enumerate(ctx):
            for j in range(counts[b]):
                self.live[self.table[b, j], :max(0, min(PAGE, n - j * PAGE))] = True
        self.codes, self.scales = {}, {}
        for c in "kv":
            self.codes[c] = np.clip(np.round(rng.normal(size=(pool, self.hkv, PAGE, self.dim)) * 3 + 8), 0, 15).astype(np.int64)
            s = rng.integers(16, 32, (pool, self.hkv, PAGE, self.dim // 32)) * 2.0 ** -6 * size      # 5 bits
            s *= rng.choice([-1.0, 1.0], s.shape) * np.exp2(np.round(rng.uniform(-spread, spread, s.shape)))
            self.scales[c] = s
        n = self.indptr[-1]
        self.q, self.kn, self.vn = bf16(rng, n, self.hq, self.dim, size=size), bf16(rng, n, self.hkv, self.dim, size=size), \
            bf16(rng, n, self.hkv, self.dim, size=size)
        self.slopes = None if slopes is None else np.asarray(slopes, np.float32)

    def cache(self):
        s = {c: np.where(self.live[:, None, :, None], self.scales[c], np.nan) for c in "kv"}
        return pack(self.codes["k"], s["k"], self.codes["v"], s["v"])

    def upload(self):
        self.d = dict(q=self.q.cuda(), cache=cu(self.cache()), k_new=self.kn.cuda(), v_new=self.vn.cuda(),
                      page_table=cu(self.table), ctx_lens=cu(self.ctx), parents=cu(self.parents))
        self.shape = native.Shape(self.indptr, self.table.shape[1], len(self.codes["k"]), window=self.window,
                                  num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.dim)
        self.out = torch.full((int(self.indptr[-1]) + 1, self.hq, self.dim), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((int(self.indptr[-1]), self.hq), 7.0, device="cuda")
        self.ws = torch.full((native.sd_kv4_attn_workspace_size(self.shape) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kw = dict(scale=self.scale, softcap=self.softcap, slopes=None if self.slopes is None else cu(self.slopes))
        return self

    def call(self, **kw):
        a = dict(workspace=self.ws, dev_status=self.status, lse=self.lse, **self.kw)
        a.update(kw)
        d = self.d
        native.sd_kv4_attn(self.shape, d["q"], d["cache"], d["k_new"], d["v_new"], d["page_table"], d["ctx_lens"], d["parents"],
                           self.out[:-1], **a)

    def ref(self, only=None):
        return kv4.attention(np64(self.q), self.cache(), np64(self.kn), np64(self.vn), self.table, self.ctx, self.indptr,
                             self.parents, scale=self.scale or None, softcap=self.softcap, slopes=self.slopes,
                             window=self.window, only=only)

    def score_error(self):
        kinf = np.abs(np64(self.kn)).max()
        for b, n in enumerate(self.ctx):
            pages = self.table[b, :-(-int(n) // PAGE)]
            if len(pages):
                kinf = max(kinf, 8 * np.abs(self.scales["k"][pages]).max())
        scale = self.scale or self.dim ** -0.5
        bias = 0.0 if self.slopes is None else 2.0 ** -23 * float(np.abs(self.slopes).max()) * (float(self.ctx.max()) + 64)
        return 2.0 ** -20 * np.abs(np64(self.q)).sum(-1).max() * kinf * scale + bias + 2.0 ** -21 * self.softcap

    def check(self, only=None):
        torch.cuda.synchronize()
        assert int(self.status) == 0
        ref, lse, spread = self.ref(only)
        at = ~np.isnan(lse)
        got, got_lse, ds = np64(self.out[:-1]), np64(self.lse), self.score_error()
        assert ds < 0.25, ds
        n = float(self.ctx.max()) + 64
        bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * np.expm1(ds) + n * 2.0 ** -27 + 2.0 ** -18) * spread + 1e-30
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
    "decode_ctx63": ([chain(1)], [63]),
    "decode_ctx65": ([chain(1)], [65]),
    "decode_ctx128": ([chain(1)], [128]),
    "decode_ctx129_narrow": ([chain(1)], [129], NARROW),
    "chain5_ctx1000": ([chain(5)], [1000]),
    "tree9_ctx513": ([tree(2, 7)], [513]),
    "tree16_ctx777": ([tree(2, 15)], [777]),
    "tree23_ctx3000": ([tree(1, 22)], [3000]),
    "tree25_ctx515": ([tree(3, 24)], [515]),
    "tree33_ctx300": ([tree(4, 32)], [300]),
    "tree64_ctx300": ([tree(4, 63)], [300]),
    "tree64_narrow_ctx4100": ([tree(4, 63)], [4100], NARROW),
    "empty_context_tree": ([tree(6, 22)], [0]),
    "ragged": ([chain(1), chain(5), tree(3, 22), chain(9), tree(4, 63)], [0, 1, 17, 700, 2049]),
    "ragged_narrow": ([chain(2), tree(5, 30), chain(1), chain(3)], [33, 1500, 0, 640], NARROW),
    "decode_batch": ([chain(1)] * 40, [(37 * i * i) % 700 for i in range(40)], NARROW),
    "decode_batch_wide": ([chain(1)] * 64, [(53 * i) % 900 for i in range(64)]),
    "chain5_batch_wide": ([chain(5)] * 40, [(71 * i) % 1300 for i in range(40)]),
    "batch_of_32": ([chain(1 + i % 3) for i in range(32)], [(83 * i) % 500 for i in range(32)], NARROW),
    "batch_of_33": ([chain(1 + i % 3) for i in range(33)], [(83 * i) % 500 for i in range(33)], NARROW),
    "batch_of_256": ([chain(1)] * 256, [(29 * i) % 300 for i in range(256)], (4, 2, 128)),
    "tree15_batch": ([tree(5, 14)] * 40, [(59 * i) % 700 for i in range(40)]),
    "tree20_batch_empty": ([tree(5, 19)] * 60, [0] * 60),
    "group1": ([tree(7, 11)], [401], (3, 3, 128)),
    "group16": ([tree(8, 6), chain(1)], [401, 90], (16, 1, 256)),
    "group5_narrow": ([tree(9, 20)], [1111], (10, 2, 128)),
    "group9_wide_nodes": ([tree(9, 63)], [200], (9, 1, 256)),
    "many_heads": ([chain(3)], [260], (64, 64, 128)),
    "long_32k": ([chain(2)], [32771], (8, 1, 256)),
}


@pytest.mark.parametrize("name", sorted(CASES, key=lambda n: sum(CASES[n][1]) * len(CASES[n][0][0])))
def test_attention_matches_oracle(name):
    c = Case(*CASES[name], seed=len(name)).upload()
    c.call()
    c.check()


MODS = {
    "window1": dict(window=1), "window7": dict(window=7), "window100": dict(window=100), "window129": dict(window=129),
    "window700": dict(window=700), "window5000": dict(window=5000), "window_largest": dict(window=2 ** 31 - 1),
    "softcap": dict(softcap=30.0), "tight_softcap": dict(softcap=0.5), "bias": dict(slopes=True),
    "bias_and_cap": dict(softcap=5.0, slopes=True), "all": dict(softcap=5.0, slopes=True, window=333), "scale": dict(scale=0.3),
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
    """Scores from nearly equal to one key taking all; scales that differ by up to 2^10 inside a token."""
    c = Case([tree(seed, 22), chain(4)], [2500, 700], seed=seed, size=size, spread=spread)
    if spread == 5.0:
        c.q = c.q / 16
    c.upload()
    c.call()
    c.check()


@pytest.mark.parametrize("step", [1.0, 12.0, 80.0])
def test_rising_scores_raise_the_reference_again_and_again(step):
    """Each tile's scores lie far above the last one's, beyond what fp32 exponentials of an old reference can hold."""
    c = Case([tree(2, 12)], [1500], seed=3)
    c.q[:] = 1.0
    c.codes["k"][:] = 9                                                    # one scale each
    for j, page in enumerate(c.table[0]):                                  # tiles come from the last to the first
        c.scales["k"][page] = kv4.round5(2.0 ** -4 * step * ((94 - j) // 8 + 1))
    c.upload()
    c.call()
    c.check()


def test_flat_background_below_a_peak():
    """One key far above thousands of equal ones: the small weights still add up."""
    for gap in (6.0, 11.0, 15.0):
        c = Case([chain(2)], [6000], (4, 1, 256), seed=4)
        c.q[:] = 0.5
        c.codes["k"][:], c.scales["k"][:] = 9, 2.0 ** -6
        c.kn[:] = 2.0 ** -6
        c.scales["k"][c.table[0, 3], 0, 5] = kv4.round5(gap / 8 + 2.0 ** -6)
        c.codes["v"][:], c.scales["v"][:] = 9, 1.0
        c.codes["v"][c.table[0, 3], 0, 5] = 7
        c.vn[:] = 1.0
        c.upload()
        c.call()
        c.check()


def test_every_code_and_extreme_scales():
    c = Case([tree(8, 22), chain(8)], [700, 333], seed=8)
    for i, x in enumerate("kv"):
        c.codes[x][:] = np.resize(np.roll(np.arange(16), 5 * i), c.codes[x].shape)
    c.scales["v"][c.table[0, 7]] = 0.0
    c.scales["k"][c.table[0, 9]] = 0.0
    c.scales["v"][c.table[0, 11]] *= 2.0 ** -90
    c.scales["k"][c.table[0, 12]] *= 2.0 ** -90
    c.upload()
    c.call()
    c.check()
    # values near bf16's largest, weighed next to nothing else
    c.scales["v"][:] = np.sign(c.scales["v"]) * 2.0 ** 110
    c.vn[:] = 0
    c.upload()
    c.call()
    c.check()


def test_scale_bits_that_do_not_count():
    """The three lowest bits of a scale are ignored."""
    a, b = (Case([tree(8, 9)], [300], seed=8) for _ in "ab")
    a.upload()
    b.upload()
    raw = b.d["cache"][..., 8 * 256:].view(torch.int16)
    raw |= torch.randint(0, 8, raw.shape, device="cuda", dtype=torch.int16)      # (a NaN stays one)
    a.call()
    b.call()
    assert torch.equal(a.out, b.out) and int(b.status) == 0


def test_masked_places_may_hold_anything():
    """NaN and infinities on other branches reach nobody who does not see them, nor do scales behind the context."""
    par = [-1, 0, 0, 1, 2, 2]
    c = Case([par], [200], seed=9)
    clean = Case([par], [200], seed=9).upload()
    clean.call()
    c.kn[1], c.vn[1], c.kn[4, 2], c.vn[5, 1, 7] = float("nan"), float("inf"), float("-inf"), float("nan")
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
    assert np.isnan(got[5, group:2 * group]).all() and np.isfinite(got[5, :group]).all()
    assert int(c.status) == 0
    # one query row of one head: an infinity makes that row NaN alone
    c = Case([par], [200], seed=9)
    c.q[2, 5, 17] = float("inf")
    c.upload()
    c.call()
    torch.cuda.synchronize()
    got = np64(c.out[:-1])
    assert np.isnan(got[2, 5]).all()
    got[2, 5] = want[2, 5]
    np.testing.assert_array_equal(got, want)
    # a window: scales of tokens before every node's window are not looked at
    c = Case([chain(4)], [500], seed=10, window=100)
    clean = Case([chain(4)], [500], seed=10, window=100).upload()
    clean.call()
    for pos in (385, 395, 400):                                             # 401 is the root's oldest position
        page, t = c.table[0, pos // PAGE], pos % PAGE
        c.scales["v"][page, :, t] = c.scales["k"][page, :, t] = np.nan
    c.table[0, 10] = -5                                                     # nor pages before it
    c.upload()
    c.call()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(np64(c.out), np64(clean.out))
    assert int(c.status) == 0


def test_bad_pages_and_scales_are_reported():
    for bad in (-1, -7, 10 ** 6):
        c = Case([tree(3, 9)], [600], seed=11)
        zero = Case([tree(3, 9)], [600], seed=11)
        page = int(c.table[0, 20])
        c.table[0, 20] = bad
        zero.scales["k"][page] = zero.scales["v"][page] = 0
        c.upload()
        zero.upload()
        c.call()
        zero.call()
        torch.cuda.synchronize()
        assert int(c.status) == native.SD_DEV_BAD_PAGE and int(zero.status) == 0
        np.testing.assert_array_equal(np64(c.out), np64(zero.out))
    for value in (float("nan"), float("inf"), -2.0 ** 125, 1.375 * 2.0 ** 123):
        for x in "kv":
            c, zero = Case([chain(3)], [600], seed=11), Case([chain(3)], [600], seed=11)
            c.scales[x][c.table[0, 3], 1, 7, 2] = value
            zero.scales[x][c.table[0, 3], 1, 7, 2] = 0.0
            for one in (c, zero):
                one.upload()
                one.call()
            torch.cuda.synchronize()
            assert int(c.status) == native.SD_DEV_BAD_SCALE and int(zero.status) == 0
            np.testing.assert_array_equal(np64(c.out), np64(zero.out))
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
    a.live[a.table[0, 111], 1:] = False          # what lies behind a shorter context
    a.live[a.table[0, 112:]] = False
    a.d["cache"].copy_(cu(a.cache()))
    a.d["ctx_lens"].fill_(1777)
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
    """The sequence's pages lie past 2^32 bytes of the pool; append and read reach them too."""
    heads, pool = (8, 4, 256), 250000                       # 18 KB a page
    c = Case([chain(3)], [1000], heads, seed=17).upload()
    far = torch.arange(pool - 70, pool - 70 + len(c.codes["k"]), device="cuda")
    big = torch.empty((pool, 4, 2, 9 * 256), dtype=torch.uint8, device="cuda")
    assert big.numel() > 2 ** 32
    big[far] = c.d["cache"]
    c.d["cache"] = big
    c.d["page_table"] = torch.where(c.d["page_table"] >= 0, c.d["page_table"] + pool - 70, -1).int()
    c.shape = native.Shape(c.indptr, c.table.shape[1], pool, num_q_heads=8, num_kv_heads=4)
    c.call()
    c.check()
    new = bf16(np.random.default_rng(1), 16, 4, 256).cuda()
    slots = torch.arange(16, dtype=torch.int32, device="cuda") + (pool - 1) * PAGE
    other = new * 3
    native.sd_kv4_append([big], [new], [other], slots)
    want = kv4.append(np.zeros((1, 4, 2, 9 * 256), np.uint8), np64(new), np64(other), range(16))
    np.testing.assert_array_equal(big[-1].cpu().numpy(), want[0])
    k, v = torch.empty_like(new), torch.empty_like(new)
    native.sd_kv4_read([big], slots, [k], [v])
    np.testing.assert_array_equal(np64(k), kv4.values(want)[0][0].transpose(1, 0, 2))


# ------------------------------------------------------------------------------------------ append and read

def run_append(cache, k, v, slots, rows=None, layers=1):
    """The calls on `layers` copies with shifted inputs; checks bytes and read-back values."""
    pool, heads, _, width = cache.shape
    dim = width // 9
    caches = cu(np.stack([cache] * layers))
    ks, vs = (torch.stack([torch.roll(x, i, 1) for i in range(layers)]) for x in (k, v))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.sd_kv4_append(caches, ks, vs, cu(slots, torch.int32), None if rows is None else cu(rows, torch.int32), status)
    k_out, v_out = (torch.full((layers, len(slots) + 1, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    read = list(slots) + [-1]
    native.sd_kv4_read(caches, cu(read, torch.int32), k_out, v_out, status)
    torch.cuda.synchronize()
    got = caches.cpu().numpy()
    for i in range(layers):
        want = kv4.append(cache, np64(ks[i]), np64(vs[i]), slots, rows)
        np.testing.assert_array_equal(got[i], want)
        for held, out in zip(kv4.values(want), (k_out[i], v_out[i])):
            out = np64(out)
            for r, s in enumerate(read):
                np.testing.assert_array_equal(out[r], held[s // PAGE, :, s % PAGE] if s >= 0 else 7.0)
    return int(status), got


def filled(rng, pool, heads, dim):
    """A cache of random bytes whose scales are numbers."""
    cache = rng.integers(0, 256, (pool, heads, 2, 9 * dim), dtype=np.uint8)
    s = cache[..., 8 * dim + 1::2]
    s[...] = (s & 0x80) | 0x3C
    return cache


@pytest.mark.parametrize("heads,dim", [(4, 256), (8, 128), (1, 256), (3, 128)])
@pytest.mark.parametrize("slots", [
    [0], [5], [15, 16 + 0], list(range(16)), list(range(3, 16)) + list(range(48, 64)) + [80, 81],
    [-1, 7, 8, -1, -1, 40, 41, 42, -1], list(range(9, 16)) + list(range(64, 72)), [-1] * 20,
], ids=["one", "one_inside", "two_pages", "page", "prompt", "gaps", "tail_and_head", "nothing"])
def test_append_and_read_match_oracle(heads, dim, slots):
    rng = np.random.default_rng(len(slots) + dim)
    cache = filled(rng, 6, heads, dim)
    size = torch.from_numpy(np.exp2(rng.uniform(-20, 20, (len(slots), heads, dim // 32, 1))).astype(np.float32))
    k, v = ((bf16(rng, len(slots), heads, dim).float().unflatten(2, (-1, 32)) * size).flatten(2).bfloat16().cuda() for _ in "kv")
    status, _ = run_append(cache, k, v, slots, layers=2)
    assert status == 0


def test_append_of_a_path():
    """Accepted nodes among others, in the order of the slot map; more rows than are used."""
    rng = np.random.default_rng(5)
    k, v = bf16(rng, 23, 4, 256).cuda(), bf16(rng, 23, 4, 256).cuda()
    assert run_append(filled(rng, 5, 4, 256), k, v, [14, 15, 64, 65, -1, -1], [0, 2, 5, 22, 0, 0], layers=16)[0] == 0


def test_a_long_prompt():
    rng = np.random.default_rng(6)
    perm = rng.permutation(40)
    slots = [int(perm[i // 16]) * 16 + i % 16 for i in range(21, 600)]
    k, v = bf16(rng, 579, 2, 256).cuda(), bf16(rng, 579, 2, 256).cuda()
    assert run_append(filled(rng, 40, 2, 256), k, v, slots)[0] == 0


def test_blocks_where_the_format_can_go_wrong():
    """Ties of magnitude, half steps, zeros, the smallest and largest, infinities and NaN."""
    rng = np.random.default_rng(7)
    x = torch.zeros(16, 1, 256)
    b = x.unflatten(2, (-1, 32))
    b[0, 0] = torch.from_numpy(rng.choice([-1.0, 1.0], (8, 32)))                        # every magnitude alike
    b[1, 0] = torch.arange(32) * 0.5 - 8                                                 # half steps on a grid of -8 .. 7.5
    b[1, 0, 1] *= -1
    b[2, 0, :, 3] = torch.tensor([2.0 ** -100, 2.0 ** -101, 2.0 ** -99, -2.0 ** -100, 1e-38, -2.0 ** -103, 0.0, -0.0])
    b[3, 0] = 3.3895313892515355e38 * torch.from_numpy(rng.choice([-1.0, 1.0, 0.4], (8, 32)))
    b[4, 0] = torch.from_numpy(rng.integers(128, 256, (8, 32)) * 2.0 ** rng.integers(-3, 3, (8, 32)))
    b[5, 0] = 8.25                                                                       # m / s = 8.25, a tie of the scale
    b[5, 0, :, 1::2] = -8.25
    b[6:9, 0] = torch.from_numpy(rng.normal(size=(3, 8, 32)))
    b[6, 0, 0, 5], b[6, 0, 1, 7], b[6, 0, 2, 0] = float("nan"), float("inf"), float("-inf")
    b[7, 0, 3] = float("inf")
    b[7, 0, 4] = float("nan")
    b[9:, 0] = torch.from_numpy(rng.integers(-255, 256, (7, 8, 32)) / 16.0)              # many half steps
    x = b.flatten(2).bfloat16().cuda()
    status, got = run_append(filled(rng, 2, 1, 256), x, x, list(range(16)))
    assert status == native.SD_DEV_NOT_FINITE
    assert run_append(filled(rng, 2, 1, 256), x[9:].contiguous(), x[9:].contiguous(), list(range(5, 12)))[0] == 0
    for held in kv4.values(got[0]):
        assert np.isfinite(held[:1]).all()


def test_slot_maps_in_the_wrong_order_are_refused():
    rng = np.random.default_rng(8)
    for slots, rows, src in (([3, 5], None, 2), ([3, 3], None, 2), ([4, 3], None, 2), ([16 * 9], None, 1), ([-2], None, 1),
                             ([3], [7], 4), ([3], [-1], 4), (list(range(16)) + [15], None, 17)):
        cache = filled(rng, 4, 2, 128)
        dev, status = cu(cache[None]), torch.zeros(1, dtype=torch.int32, device="cuda")
        new = bf16(rng, src, 2, 128).cuda()
        native.sd_kv4_append(dev, new[None], new[None], cu(slots, torch.int32), None if rows is None else cu(rows, torch.int32), status)
        assert int(status) == native.SD_DEV_BAD_SLOT
        np.testing.assert_array_equal(dev[0].cpu().numpy(), cache)


def test_read_in_any_order():
    rng = np.random.default_rng(9)
    cache = filled(rng, 7, 3, 256)
    slots = rng.integers(-1, 7 * 16, 200).tolist() + [3, 3, 3]
    out = torch.full((203, 8, 256), 7.0, dtype=torch.bfloat16, device="cuda")          # rows that lie apart
    k, v = out[:, :3], out[:, 4:7]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.sd_kv4_read([cu(cache)], cu(slots, torch.int32), [k], [v], status)
    for held, got in zip(kv4.values(cache), (np64(k), np64(v))):
        for r, s in enumerate(slots):
            np.testing.assert_array_equal(got[r], held[s // 16, :, s % 16] if s >= 0 else 7.0)
    assert int(status) == 0 and torch.all(out[:, 3] == 7.0) and torch.all(out[:, 7] == 7.0)
    cache[2, 1, :, 8 * 256 + 1::2] |= 0x7F                                               # infinities and NaN
    native.sd_kv4_read([cu(cache)], cu([40, 7 * 16, -9, 3], torch.int32), [k[:4]], [v[:4]], status)
    assert int(status) == native.SD_DEV_BAD_SCALE | native.SD_DEV_BAD_SLOT
    assert np.array_equal(np64(k[0, 1]), np.zeros(256)) and np.array_equal(np64(v[3]), kv4.values(cache)[1][0, :, 3])


def test_append_and_read_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(10)
    cache = filled(rng, 6, 4, 256)
    slots = list(range(7, 16)) + list(range(32, 48))
    k, v = bf16(rng, 25, 4, 256).cuda(), bf16(rng, 25, 4, 256).cuda()
    dev, at = cu(cache), cu(slots, torch.int32)
    k_out, v_out = torch.empty_like(k), torch.empty_like(v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        native.sd_kv4_append([dev], [k], [v], at)
        native.sd_kv4_read([dev], at, [k_out], [v_out])
    for seed in (11, 12):
        k.copy_(bf16(np.random.default_rng(seed), 25, 4, 256))
        g.replay()
        torch.cuda.synchronize()
        want = kv4.append(cache, np64(k), np64(v), slots)
        np.testing.assert_array_equal(dev.cpu().numpy(), want)
        np.testing.assert_array_equal(np64(k_out)[3], kv4.values(want)[0][0, :, 10])


@pytest.mark.parametrize("heads", [(24, 4, 256), (8, 2, 128)], ids=["d256", "d128"])
@pytest.mark.parametrize("q_power,k_power", [(0, 100), (60, 30), (0, 30), (20, 10), (100, 0), (12, 12)])
@pytest.mark.parametrize("nodes", [1, 23])
def test_scores_so_large_that_one_key_is_left(nodes, q_power, k_power, heads):
    """Scores of 2^24 to 2^110: softmax leaves the largest alone (its nearest rival is farther off than fp32's rounding of
    either, else the column is passed over), so the output is that key's value, which bf16 holds exactly."""
    c = Case([chain(nodes), chain(nodes)], [700, 5], heads, seed=31, spread=0.0)
    c.q = (c.q.float() * 2.0 ** q_power).bfloat16()
    c.scales["k"] = c.scales["k"] * 2.0 ** k_power
    c.kn = (c.kn.float() * 2.0 ** k_power).bfloat16()
    c.upload().call()
    torch.cuda.synchronize()
    assert int(c.status) == 0
    got, lse = np64(c.out[:-1]), np64(c.lse)
    assert np.isfinite(got).all() and np.isfinite(lse).all()
    k, v = kv4.values(c.cache())
    q, kn, vn, seen = np64(c.q), np64(c.kn), np64(c.vn), 0
    for b in range(2):
        pages = c.table[b, :-(-int(c.ctx[b]) // PAGE)]
        for j in range(nodes):
            r = c.indptr[b] + j
            for h in range(c.hq):
                g = h // (c.hq // c.hkv)
                flat = lambda x, new: np.concatenate([x[pages, g].reshape(-1, c.dim)[:c.ctx[b]], new[c.indptr[b]:r + 1, g]])
                keys, vals = flat(k, kn), flat(v, vn)
                s = keys @ q[r, h] * c.dim ** -0.5
                top = np.argmax(s)
                off = 2.0 ** -20 * np.abs(keys).max() * np.abs(q[r, h]).sum() * c.dim ** -0.5 + 2.0 ** -22 * np.abs(s[top])
                if np.sort(s)[-2] + 2 * off + 40 < s[top]:        # e^-40 of all others is nothing
                    seen += 1
                    np.testing.assert_array_equal(got[r, h], vals[top])
                    assert abs(lse[r, h] - s[top]) <= off + 2.0 ** -20 * np.abs(s[top])
    assert seen > 10
