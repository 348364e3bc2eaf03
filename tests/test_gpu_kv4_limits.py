"""The ends of what include/sd_kv4.h promises: values as large as the attention's sums can hold, infinities in an append."""
import numpy as np
import pytest
import torch

import oracle.kv4_oracle as kv4
from speculative_decoding_verify_decode_gb300 import native

from gpu_helpers import ensure_built
from test_gpu_kv4 import Case, chain, filled, run_append

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


@pytest.mark.parametrize("heads", [(4, 1, 256), (4, 1, 128)], ids=["d256", "d128"])
@pytest.mark.parametrize("nodes", [1, 5, 23, 36])
def test_values_as_large_as_sums_can_hold(nodes, heads):
    """n keys of n |v| just below 2^112, all of one sign, whose weights come to nearly 2^16 of the reference that a piece's
    first tile gives it: sums of up to 2^128.  The mean is v itself."""
    L, dim = 4000, heads[2]
    batch = 150                                                             # pieces of many tiles
    c = Case([chain(nodes)] * batch, [L] + [0] * (batch - 1), heads, seed=21, max_pages=L // 16)
    c.ctx[:], c.table[:] = L, c.table[0]                                    # every sequence reads the same pages
    c.q[:], c.kn[:] = 1.0, 0.0
    c.codes["k"][:], c.scales["k"][:] = 9, 0.0
    rise = kv4.round5(15.8 / (dim ** 0.5 * np.log2(np.e)))                  # (5 bits of it: 15.81 and 15.87 in base 2)
    assert 15.5 < rise * dim ** 0.5 * np.log2(np.e) < 16.0
    high = [p for j, p in enumerate(c.table[0]) if (j // 64) % 2 == 0]      # tokens 0 to 1023 and 2048 to 3071
    c.scales["k"][high] = rise
    v = -2.0 ** 100 * (1 - 2.0 ** -8)                                       # in 8 bits
    c.codes["v"][:], c.scales["v"][:] = 0, kv4.round5(15.5 * 2.0 ** 93)
    held = -8.0 * kv4.round5(15.5 * 2.0 ** 93)
    assert held == -15.5 * 2.0 ** 96
    c.vn[:] = v
    assert 2.0 ** 111 < (L + nodes) * abs(v) < 2.0 ** 112 and abs(held) < abs(v)
    c.upload()
    c.call()
    torch.cuda.synchronize()
    assert int(c.status) == 0
    c.check(only={(0, 0), (nodes - 1, 3), (77 * nodes, 1), (batch * nodes - 1, 2)})
    assert torch.isfinite(c.out[:-1]).all() and torch.isfinite(c.lse).all()


@pytest.mark.parametrize("heads,nodes", [((4, 1, 256), 1), ((4, 1, 128), 1), ((6, 1, 256), 5), ((6, 1, 128), 23)])
def test_sums_over_a_million_keys(heads, nodes):
    """Values of one sign over 2^20 keys, in pieces of nearly as many: sums lose 16 keys' step by step at most 2^-23 of themselves.
    The context is 64 pages again and again, so that the reference is a sum over those.  Tolerance as in test_gpu_kv4.py."""
    batch, L, pages = 152, 1 << 20, 64
    hq, hkv, dim = heads
    c = Case([chain(nodes)] * batch, [pages * 16] + [0] * (batch - 1), heads, seed=23, size=0.5, spread=0.0)
    rng = np.random.default_rng(23)
    c.codes["v"], c.scales["v"] = rng.integers(9, 16, c.codes["v"].shape), np.abs(c.scales["v"])
    c.vn = c.vn.abs()
    table = torch.from_numpy(c.table[0, :pages].copy()).cuda()
    c.ctx[:] = L
    c.table = np.full((batch, 1), -1, np.int32)
    c.upload()
    c.d["page_table"] = table.repeat(L // (16 * pages))[None].repeat(batch, 1).contiguous()
    c.shape = native.Shape(c.indptr, L // 16, len(c.codes["k"]), num_q_heads=hq, num_kv_heads=hkv, head_dim=dim)
    c.ws = torch.empty(native.sd_kv4_attn_workspace_size(c.shape), dtype=torch.uint8, device="cuda")
    c.call()
    torch.cuda.synchronize()
    assert int(c.status) == 0
    k, v = (torch.from_numpy(x[c.d["page_table"][0, :pages].cpu().numpy(), 0].reshape(-1, dim)).cuda() for x in kv4.values(c.cache()))
    last = torch.arange(1, batch + 1, device="cuda") * nodes - 1              # the nodes that see all of their sequence's
    q, kn, vn = (c.d[x].double() for x in ("q", "k_new", "v_new"))
    kn, vn = (x[:, 0].unflatten(0, (batch, nodes)) for x in (kn, vn))
    s = torch.cat([torch.einsum("bhd,kd->bhk", q[last], k), torch.einsum("bhd,bkd->bhk", q[last], kn)], 2) * dim ** -0.5
    s[:, :, :16 * pages] += np.log(L / (16 * pages))
    p = torch.softmax(s, 2)
    ref = torch.einsum("bhk,kd->bhd", p[:, :, :16 * pages], v) + torch.einsum("bhk,bkd->bhd", p[:, :, 16 * pages:], vn)
    ds = c.score_error()
    assert ds < 0.25
    bound = (2.0 ** -8 + 2.0 ** -8 + 2 * np.expm1(ds) + (L + nodes) * 2.0 ** -27 + 2.0 ** -18) * ref       # ref > 0: it is the spread as well
    assert torch.all((c.out[:-1][last].double() - ref).abs() <= bound)
    lse = torch.logsumexp(s, 2)
    assert torch.all((c.lse[last].double() - lse).abs() <= ds + 2.0 ** -20 * (lse.abs() + 1))


def test_infinities_in_blocks_without_a_range():
    """Blocks of infinities, NaN and values below 2^-100 are held as 0; from 2^-100 on infinities are the ends of the range."""
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(16, 2, 128)
    b = x.unflatten(2, (-1, 32))
    b[0, 0] = inf
    b[1, 0] = -inf
    b[2, 0, :, ::2], b[2, 0, :, 1::2] = inf, nan
    b[3, 0, 0, 5], b[3, 0, 1, 31], b[3, 0, 2, 0] = inf, -inf, nan                      # others 0
    b[4, 0] = 2.0 ** -101
    b[4, 0, :, 7], b[4, 0, :, 8] = inf, -inf
    b[5, 0] = -2.0 ** -101 * (2 - 2.0 ** -7)
    b[5, 0, 1, 3] = inf
    b[6, 0] = 2.0 ** -100
    b[6, 0, :, 7], b[6, 0, :, 8] = inf, -inf
    b[7, 0] = -2.0 ** -100
    b[7, 0, 2, 7], b[7, 0, 3, 8] = inf, nan
    x = x.bfloat16().cuda()
    cache = filled(np.random.default_rng(3), 2, 2, 128)
    status, got = run_append(cache, x, x.flip(0).contiguous(), list(range(16)))
    assert status == native.SD_DEV_NOT_FINITE
    k = kv4.values(got[0])[0][0, 0]
    assert not k[:6].any()
    np.testing.assert_array_equal(k[6].reshape(4, 32)[:, 6:9], np.tile([2.0 ** -100, 2.0 ** -100, -0.875 * 2.0 ** -100], (4, 1)))
    assert k[7, 64 + 7] == 0.875 * 2.0 ** -100 and k[7, 96 + 8] == 0.0
