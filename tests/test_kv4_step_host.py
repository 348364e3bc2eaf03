"""Host logic of Kv4Cache, Kv4Step and rope_table, on the CPU: the library's calls are replaced by the oracle or by recorders."""
import math

import numpy as np
import torch

import oracle.kv4_oracle as kv4
import oracle.kv8_oracle as kv8
import oracle.token_oracle as tok
from speculative_decoding_verify_decode_gb300 import native
from speculative_decoding_verify_decode_gb300.step import Kv4Cache, Kv4Step, rope_table


def test_table_keeps_the_digits_of_far_positions():
    t = rope_table(70000, 8, theta=100.0, device="cpu")
    assert t.shape == (70000, 8) and t.dtype == torch.float32 and t.is_contiguous()
    for p in (0, 1, 511, 69999):
        for i in range(4):
            a = p * 100.0 ** (-2 * i / 8)
            assert abs(float(t[p, i]) - math.cos(a)) <= 2.0 ** -24 and abs(float(t[p, 4 + i]) - math.sin(a)) <= 2.0 ** -24
    x = np.random.default_rng(0).normal(size=(1, 1, 8))
    np.testing.assert_allclose(np.linalg.norm(tok.rotate(x, t.double().numpy(), [69999])), np.linalg.norm(x), rtol=1e-6)


def _extend(ctx_lens, add, table, held, new_held, free_list, count, new_count, slots, rows=None, new_ctx_lens=None, q_indptr=None,
            path=None, dev_status=None, stream=None):
    """sd_pages_extend as its header states it, on CPU tensors."""
    t, h, f, sl, rw, _, ctx = kv8.pages_extend(ctx_lens.tolist(), add.tolist(), table.numpy(), held.tolist(),
                                               free_list[:int(count)].tolist(), slots.numel(), q_indptr,
                                               None if path is None else path.tolist())
    table.copy_(torch.from_numpy(np.asarray(t)))
    new_held.copy_(torch.tensor(h))
    new_count.fill_(len(f))
    new_ctx_lens.copy_(torch.tensor(ctx))
    slots.copy_(torch.tensor(sl))
    if rows is not None:
        rows.copy_(torch.tensor(rw))


def _append(caches, k, v, slots, rows, status):
    for c, kk, vv in zip(caches, k, v):
        c.copy_(torch.from_numpy(kv4.append(c.numpy(), kk.double().numpy(), vv.double().numpy(), slots.tolist(),
                                            None if rows is None else rows.tolist())))


def test_extend_takes_pages_and_appends(monkeypatch):
    monkeypatch.setattr(native, "sd_pages_extend", _extend)
    monkeypatch.setattr(native, "sd_kv4_append", _append)
    c = Kv4Cache(2, 8, 12, 2, num_kv_heads=1, head_dim=128, device="cpu")
    x = torch.randn(2, 40, 1, 128).bfloat16()
    slots = torch.empty(40, dtype=torch.int32)
    c.extend(torch.tensor([30, 10], dtype=torch.int32), x, x, slots)
    assert c.ctx_lens.tolist() == [30, 10] and c.held.tolist() == [2, 1] and int(c.free_count) == 9
    for layer in range(2):
        k, v = (y.transpose(0, 2, 1, 3).reshape(-1, 1, 128) for y in kv4.values(c.kv[layer].numpy()))
        np.testing.assert_array_equal(k[slots.tolist()], v[slots.tolist()])
        for r, s in enumerate(slots.tolist()):
            for b in range(4):
                codes, scale = kv4.quantise(x[layer, r, 0, 32 * b:32 * b + 32].double().numpy())
                np.testing.assert_array_equal(k[s, 0, 32 * b:32 * b + 32], (codes - 8) * scale)


def test_a_steps_calls_in_their_order(monkeypatch):
    calls = []
    monkeypatch.setattr(native, "sd_kv4_attn_workspace_size", lambda shape: 64)
    monkeypatch.setattr(native, "sd_accept_workspace_size", lambda indptr, vocab: 64)
    for name in ("sd_rope_append", "sd_kv4_attn", "sd_accept", "sd_pages_extend", "sd_kv4_append", "sd_logprobs", "sd_kv8_attn"):
        monkeypatch.setattr(native, name, lambda *a, name=name, **kw: calls.append((name, a, kw)))
    c = Kv4Cache(2, 8, 16, 2, num_kv_heads=1, head_dim=128, device="cpu")

    class Current:
        def __init__(self, device):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *_):
            pass

    monkeypatch.setattr(torch.cuda, "device", Current)
    one = lambda heads: torch.zeros(2, 4, heads, 128, dtype=torch.bfloat16)
    ints = torch.zeros(4, dtype=torch.int32)
    names = lambda: [n for n, *_ in calls]
    whole = ["sd_kv4_attn", "sd_kv4_attn", "sd_accept", "sd_pages_extend", "sd_kv4_append"]
    Kv4Step(c, [0, 3, 4], 50, num_q_heads=2).run(one(2), one(1), one(1), ints, ints, torch.zeros(4, 50))
    assert names() == whole
    calls.clear()
    step = Kv4Step(c, [0, 3, 4], 50, num_q_heads=2, top=3)
    k = one(1)
    step.run(one(2), k, one(1), ints, ints, torch.zeros(4, 50), rope=(rope_table(9, 64, device="cpu"), ints))
    assert names() == ["sd_rope_append"] * 2 + whole + ["sd_logprobs"]
    # the attention and the append get the turned keys, the log probabilities the step's own choices
    assert calls[2][1][1].data_ptr() == step.q_turned.data_ptr() and calls[2][1][3].data_ptr() == step.k_turned.data_ptr()
    assert calls[6][1][1].data_ptr() == step.k_turned.data_ptr()
    assert calls[7][1][1].data_ptr() == step.target_tokens.data_ptr() and calls[7][1][1].shape == (4, 1)
