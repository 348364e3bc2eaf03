"""Host logic of Kv8Cache and Kv8Step, on the CPU: the library's calls are replaced by the oracle or by recorders."""
import numpy as np
import pytest
import torch

import oracle.kv8_oracle as kv8
from speculative_decoding_verify_decode_gb300 import native
from speculative_decoding_verify_decode_gb300.step import Kv8Cache, Kv8Step


def _release(keep, table, held, new_held, free_list, count, new_count, status=None, stream=None):
    """sd_pages_release as its header states it, on CPU tensors."""
    k, h, n, pool = keep.tolist(), held.tolist(), int(count), free_list.numel()
    bad = native.SD_DEV_BAD_CTX if any(x < 0 for x in k) or any(not 0 <= x <= table.shape[1] for x in h) else 0
    left, free = kv8.pages_release(k, table.numpy(), h, free_list[:max(n, 0)].tolist()) if not bad else (h, [])
    if not bad and not 0 <= n <= len(free) <= pool:
        bad = native.SD_DEV_BAD_PAGE
    new_held.copy_(torch.tensor(h if bad else left))
    new_count.fill_(n if bad else len(free))
    if not bad:
        free_list[:len(free)] = torch.tensor(free, dtype=torch.int32)
        bad = native.SD_DEV_BAD_PAGE if any(not 0 <= x < pool for x in free[n:]) else 0
    status |= bad


@pytest.mark.parametrize("plant,keep,want", [
    (None, [10, 100], [10, 20]), (None, [50, 17], [50, 17]), (None, [10, -1], None),
    (lambda c: c.held.__setitem__(1, 9), [10, 20], None), (lambda c: c.free_count.fill_(16), [10, 20], None),
    (lambda c: c.page_table.__setitem__((0, 2), 99), [10, 20], [10, 20]),
])
def test_release_moves_contexts_only_when_pages_may_move(monkeypatch, plant, keep, want):
    monkeypatch.setattr(native, "sd_pages_release", _release)
    c = Kv8Cache(2, 8, 16, 1, num_kv_heads=1, head_dim=128, device="cpu")
    table, held, free, *_, ctx = kv8.pages_extend([0, 0], [50, 20], c.page_table.numpy(), [0, 0], c.free_list.tolist(), 70)
    c.page_table.copy_(torch.from_numpy(np.asarray(table)))
    c.held.copy_(torch.tensor(held))
    c.ctx_lens.copy_(torch.tensor(ctx))
    c.free_count.fill_(len(free))
    if plant:
        plant(c)
    before = c.held.clone(), c.free_count.clone()
    c.dev_status.fill_(native.SD_DEV_BAD_ACCEPT)            # of an earlier call
    c.release(torch.tensor(keep, dtype=torch.int32))
    assert c.ctx_lens.tolist() == (ctx if want is None else want)
    assert int(c.dev_status) & native.SD_DEV_BAD_ACCEPT
    if want is None:
        assert torch.equal(c.held, before[0]) and torch.equal(c.free_count, before[1])
        assert int(c.dev_status) & ~native.SD_DEV_BAD_ACCEPT


def test_a_step_runs_on_its_caches_device(monkeypatch):
    """sd_accept goes by the current device, so a step makes its cache's device current."""
    now, calls = [None], []

    class Current:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, now[0] = now[0], self.device

        def __exit__(self, *_):
            now[0] = self.before

    c = Kv8Cache(2, 8, 16, 2, num_kv_heads=1, head_dim=128, device="cpu")
    monkeypatch.setattr(native, "sd_kv8_attn_workspace_size", lambda shape: 64)
    monkeypatch.setattr(native, "sd_accept_workspace_size", lambda indptr, vocab: 64)
    for name in ("sd_kv8_attn", "sd_accept", "sd_pages_extend", "sd_kv8_append"):
        monkeypatch.setattr(native, name, lambda *a, name=name, **kw: calls.append((name, now[0])))
    step = Kv8Step(c, [0, 3, 4], 50, num_q_heads=2)
    monkeypatch.setattr(torch.cuda, "device", Current)
    one = lambda heads: torch.zeros(2, 4, heads, 128, dtype=torch.bfloat16)
    ints = torch.zeros(4, dtype=torch.int32)
    step.run(one(2), one(1), one(1), ints, ints, torch.zeros(4, 50))
    assert calls == [(n, c.k.device) for n in ("sd_kv8_attn", "sd_kv8_attn", "sd_accept", "sd_pages_extend", "sd_kv8_append")]
    assert c.device == c.k.device and now == [None]
