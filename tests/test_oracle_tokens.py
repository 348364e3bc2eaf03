"""Pins of the oracle of rotation, append and log probabilities."""
import math

import numpy as np
import pytest
import torch

import oracle.token_oracle as tok


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_one(inter):
    """Norms stay, position 0 changes nothing, angles add up, and q.k depends on the distance alone."""
    rng = np.random.default_rng(1)
    freq = 10.0 ** -rng.uniform(0, 3, 4)
    angle = np.arange(50)[:, None] * freq
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    x, y = rng.normal(size=(2, 3, 12)), rng.normal(size=(2, 3, 12))
    np.testing.assert_array_equal(tok.rotate(x, table, [0, 0], inter), x)
    a = tok.rotate(x, table, [7, 9], inter)
    np.testing.assert_allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1))
    np.testing.assert_array_equal(a[..., 8:], x[..., 8:])                            # the rest does not turn
    np.testing.assert_allclose(tok.rotate(a, table, [5, 5], inter), tok.rotate(x, table, [12, 14], inter))
    dot = lambda p, q: (tok.rotate(x, table, [p, p], inter) * tok.rotate(y, table, [q, q], inter)).sum(-1)
    np.testing.assert_allclose(dot(3, 10), dot(23, 30))


def test_rotation_pairs():
    x = np.zeros((1, 1, 8))
    x[0, 0, 1] = 1.0
    table = np.array([[1.0, 0.0, 1.0, 1.0, 0.0, 1.0, 0.0, 0.0]])                      # pair 1 turns by a right angle
    assert np.argmax(np.abs(tok.rotate(x, table, [0])[0, 0])) == 5                    # dim 1 with dim 1 + 4
    assert np.argmax(np.abs(tok.rotate(np.roll(x, 1, -1), table, [0], True)[0, 0])) == 3   # dim 2 with dim 3


def test_put():
    cache, rows = np.zeros((3, 2, 16, 4)), np.arange(24.0).reshape(3, 2, 4) + 1
    got = tok.put(cache, rows, [33, -1, 7])
    np.testing.assert_array_equal(got[2, :, 1], rows[0])
    np.testing.assert_array_equal(got[0, :, 7], rows[2])
    assert (got != 0).sum() == 16


def test_logprobs_against_torch():
    g = torch.Generator().manual_seed(1)
    for t in (1.0, 0.3, 2.0):
        x = torch.randn(501, generator=g, dtype=torch.float64) * 4
        x[17] = x[3]
        given, ids, best, entropy, lse = tok.logprobs(x.tolist(), [0, 17, 501, -1], 20, t)
        p = torch.log_softmax(x / t, 0)
        assert given[:2] == pytest.approx([float(p[0]), float(p[17])], rel=1e-12) and given[2:] == [-math.inf] * 2
        assert ids == torch.sort(x, descending=True, stable=True)[1][:20].tolist()
        assert best == pytest.approx(p[ids].tolist(), rel=1e-12)
        assert entropy == pytest.approx(float(-(p.exp() * p).sum()), rel=1e-11) and lse == pytest.approx(float(torch.logsumexp(x / t, 0)))


def test_logprobs_by_hand():
    given, ids, best, entropy, lse = tok.logprobs([0.0, -math.inf, 0.0, -0.0], [1, 3], 4, 1.0)
    assert ids == [0, 2, 3, 1] and best[3] == -math.inf and given[0] == -math.inf
    assert entropy == pytest.approx(math.log(3)) and lse == pytest.approx(math.log(3)) and given[1] == pytest.approx(-math.log(3))
    assert tok.logprobs([-math.inf] * 3, [0], 2) == ([-math.inf], [0, 1], [-math.inf] * 2, 0.0, -math.inf)
    given, _, best, entropy, _ = tok.logprobs([40.0, 0.0], [0, 1], 1)                  # far below 1's steps
    assert best[0] == pytest.approx(-math.exp(-40), rel=1e-12) and entropy == pytest.approx(41 * math.exp(-40), rel=1e-12)
