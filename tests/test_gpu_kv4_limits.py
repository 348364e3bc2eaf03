"""The ends of what include/sd_kv4.h promises: values as large as the attention's sums can hold."""
import numpy as np
import pytest
import torch

import oracle.kv4_oracle as kv4

from gpu_helpers import ensure_built
from test_gpu_kv4 import Case, chain

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
