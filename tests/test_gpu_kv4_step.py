"""Whole verify steps over the 4-bit cache on the GPU: rotation, attention, accept, pages, append and log probabilities together,
every part against its oracle (tolerances as in the tests of the parts)."""
import numpy as np
import pytest
import torch

import oracle
import oracle.kv4_oracle as kv4
import oracle.kv8_oracle as kv8
from speculative_decoding_verify_decode_gb300 import native
from speculative_decoding_verify_decode_gb300.step import Kv4Cache, Kv4Step, rope_table

from gpu_helpers import ensure_built
from test_gpu_kv4 import bf16, chain, cu, np64, tree
from test_gpu_tokens import check as check_logprobs, near_rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


def depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def near_attention(got, q, kn, vn, cache, table, ctx, indptr, parents, softcap):
    ref, _, spread = kv4.attention(np64(q), cache, np64(kn), np64(vn), table, ctx, indptr, parents, softcap=softcap)
    dim = q.shape[-1]
    kinf = max(np.abs(np64(kn)).max(), max(np.abs(kv4.values(cache)[0]).max(), 0))
    ds = 2.0 ** -20 * np.abs(np64(q)).sum(-1).max() * kinf * dim ** -0.5 + 2.0 ** -21 * softcap
    assert ds < 0.25
    n = max(ctx) + 64
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * np.expm1(ds) + n * 2.0 ** -27 + 2.0 ** -18) * spread + 1e-30
    assert np.all(np.abs(np64(got) - ref) <= bound)


@pytest.mark.parametrize("hq,heads,dim,rot", [(24, 4, 256, 64), (32, 8, 128, 128)], ids=["d256", "d128"])
@pytest.mark.parametrize("how", ["eager", "graph", "side_stream"])
def test_prompt_then_verify_steps(how, hq, heads, dim, rot):
    layers, vocab, top, batch = 2, 9001, 5, 3
    par = [tree(1, 10), chain(4), chain(1)]
    indptr = np.cumsum([0] + [len(p) for p in par])
    parents, total = np.concatenate(par).astype(np.int32), int(indptr[-1])
    depth = np.concatenate([depths(p) for p in par])
    cache = Kv4Cache(batch, 40, 64, layers, num_kv_heads=heads, head_dim=dim)
    step = Kv4Step(cache, indptr, vocab, num_q_heads=hq, softcap=20.0, top=top)
    table_r = rope_table(1024, rot)
    rng = np.random.default_rng(3)
    side = torch.cuda.Stream() if how == "side_stream" else None

    # the prompts: turned, then appended
    lens = [200, 31, 0]
    where = cu(np.concatenate([np.arange(n) for n in lens + [240 - sum(lens)]]), torch.int32)
    prompt = [[bf16(rng, 240, heads, dim).cuda() for _ in range(layers)] for _ in "kv"]
    turned = [torch.empty_like(x) for x in prompt[0]]
    for x, y in zip(prompt[0], turned):
        native.sd_rope_append(table_r, where, k=x, k_out=y, dev_status=cache.dev_status)
        near_rotated(y, x, table_r, where.tolist(), False)
    slots = torch.empty(240, dtype=torch.int32, device="cuda")
    cache.extend(cu(lens, torch.int32), turned, prompt[1], slots)
    table, held, free, sl, _, _, ctx = kv8.pages_extend([0] * batch, lens, np.full((batch, 40), -1), [0] * batch,
                                                        list(range(63, -1, -1)), 240)
    pages = [kv4.append(np.zeros(cache.kv.shape[1:], np.uint8), np64(k), np64(v), sl) for k, v in zip(turned, prompt[1])]
    np.testing.assert_array_equal(cache.kv.cpu().numpy(), np.stack(pages))
    kr, vr = ([torch.empty(200, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(layers)] for _ in "kv")
    cache.read(cu(sl[:200], torch.int32), kr, vr)
    for layer in range(layers):
        vk, vv = (x.transpose(0, 2, 1, 3).reshape(-1, heads, dim)[sl[:200]] for x in kv4.values(pages[layer]))
        np.testing.assert_array_equal(np64(kr[layer]), vk)
        np.testing.assert_array_equal(np64(vr[layer]), vv)

    buf = dict(q=torch.empty(layers, total, hq, dim, dtype=torch.bfloat16, device="cuda"),
               k=torch.empty(layers, total, heads, dim, dtype=torch.bfloat16, device="cuda"),
               v=torch.empty(layers, total, heads, dim, dtype=torch.bfloat16, device="cuda"),
               logits=torch.empty(total, vocab, device="cuda"), draft=torch.zeros(total, dtype=torch.int32, device="cuda"),
               pos=torch.zeros(total, dtype=torch.int32, device="cuda"), par=cu(parents))
    run = lambda: step.run(buf["q"], buf["k"], buf["v"], buf["par"], buf["draft"], buf["logits"], side,
                           rope=(table_r, buf["pos"]))
    graph = None
    for _ in range(3):
        buf["q"].copy_(bf16(rng, *buf["q"].shape))
        buf["k"].copy_(bf16(rng, *buf["k"].shape))
        buf["v"].copy_(bf16(rng, *buf["v"].shape))
        logits = (rng.normal(size=(total, vocab)) * 3).astype(np.float32)
        t = logits.argmax(1)
        draft = np.array([0 if parents[r] < 0 else (t[indptr[b] + parents[r]] if rng.random() < 0.8 else 1 + t[r] % 5)
                          for b in range(batch) for r in range(indptr[b], indptr[b + 1])], np.int32)
        buf["logits"].copy_(torch.from_numpy(logits))
        buf["draft"].copy_(torch.from_numpy(draft))
        pos = depth + np.repeat(ctx, np.diff(indptr))
        buf["pos"].copy_(torch.from_numpy(pos))
        if how == "graph" and graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
        if side:
            side.wait_stream(torch.cuda.current_stream())
        graph.replay() if graph else run()
        torch.cuda.synchronize()
        assert int(cache.dev_status) == 0
        _, alen, paths, _ = oracle.accept(indptr, parents, draft, logits)
        assert step.accept_len.tolist() == list(alen)
        for layer in range(layers):
            near_rotated(step.q_turned[layer], buf["q"][layer], table_r, pos, False)
            near_rotated(step.k_turned[layer], buf["k"][layer], table_r, pos, False)
            near_attention(step.out[layer], step.q_turned[layer], step.k_turned[layer], buf["v"][layer], pages[layer], table, ctx,
                           indptr, parents, 20.0)
        table, held, free, sl, rows, _, ctx = kv8.pages_extend(ctx, alen, table, held, free, total, indptr, paths)
        assert step.slots.tolist() == sl and step.rows.tolist() == rows
        pages = [kv4.append(c, np64(k), np64(v), sl, rows) for c, k, v in zip(pages, step.k_turned, buf["v"])]
        np.testing.assert_array_equal(cache.kv.cpu().numpy(), np.stack(pages))
        assert step.target_tokens.tolist() == list(t)
        check_logprobs(buf["logits"], dict(tokens=step.target_tokens[:, None], logprobs=step.logprobs, top_ids=step.top_ids,
                                           top_logprobs=step.top_logprobs, entropy=step.entropy,
                                           lse=torch.logsumexp(buf["logits"].double(), 1)))
        assert torch.equal(step.logprobs[:, 0], step.top_logprobs[:, 0])
        assert cache.ctx_lens.tolist() == list(ctx) and cache.held.tolist() == list(held)
    cache.release(cu([100, 0, 10 ** 6], torch.int32))
    held, free = kv8.pages_release([100, 0, 10 ** 6], table, held, free)
    assert cache.held.tolist() == held and int(cache.free_count) == len(free)


def test_a_rotating_append_into_the_bf16_cache_then_its_attention():
    """The bf16 path's own verify attention reads what sd_rope_append has put into the cache."""
    hq, heads, dim, rot, ctx, nodes = 24, 4, 256, 256, 75, 4
    rng = np.random.default_rng(8)
    table_r = rope_table(256, rot)
    k, v = bf16(rng, ctx, heads, dim).cuda(), bf16(rng, ctx, heads, dim).cuda()
    kc, vc = (torch.zeros(6, heads, 16, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    order = [4, 0, 5, 2, 1]
    slots = cu([order[t // 16] * 16 + t % 16 for t in range(ctx)], torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.sd_rope_append(table_r, cu(range(ctx), torch.int32), k=k, v=v, k_cache=kc, v_cache=vc, slots=slots, dev_status=status)
    q, kn, vn = bf16(rng, nodes, hq, dim).cuda(), bf16(rng, nodes, heads, dim).cuda(), bf16(rng, nodes, heads, dim).cuda()
    native.sd_rope_append(table_r, cu(range(ctx, ctx + nodes), torch.int32), q=q, k=kn, q_out=q, k_out=kn, dev_status=status)
    shape = native.Shape([0, nodes], 5, 6, num_q_heads=hq, num_kv_heads=heads, head_dim=dim)
    out = torch.empty_like(q)
    ws = torch.empty(max(16, native.sd_verify_attn_workspace_size(shape)), dtype=torch.uint8, device="cuda")
    native.sd_verify_attn(shape, q, kc, vc, kn, vn, cu([order], torch.int32), cu([ctx], torch.int32), cu(chain(nodes), torch.int32),
                          out, workspace=ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    at = slots.long()
    keys = torch.cat([kc[at // 16, :, at % 16], kn]).double().repeat_interleave(6, 1).transpose(0, 1)
    vals = torch.cat([vc[at // 16, :, at % 16], vn]).double().repeat_interleave(6, 1).transpose(0, 1)
    mask = torch.ones(nodes, ctx + nodes, dtype=torch.bool, device="cuda").tril(ctx)
    s = (q.double().transpose(0, 1) @ keys.transpose(1, 2) * dim ** -0.5).masked_fill(~mask, -torch.inf).softmax(-1)
    ref = (s @ vals).transpose(0, 1)
    spread = (s @ vals.abs()).transpose(0, 1)
    # bf16 output and bf16 weights, half a step each, and 2^-8 more for scores and sums in fp32
    assert torch.all((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -7 * spread)


def test_all_the_attentions_one_after_the_other():
    """bf16, 4-bit and 8-bit attention, rotation, appends and log probabilities in one stream and one graph, each launched while
    the one before drains: the same bits as alone."""
    from test_gpu_kv4 import Case
    from test_gpu_kv8 import Case as Case8
    heads, dim, rng = (24, 4, 256), 256, np.random.default_rng(11)
    small, wide = Case([chain(1)], [700], heads, seed=1).upload(), Case([tree(2, 22), chain(2)], [9000, 40], heads, seed=2).upload()
    eight = Case8([tree(3, 12)], [3000], heads, seed=3).upload()
    pages, nodes = 40, 9
    kc, vc = bf16(rng, pages, 4, 16, dim).cuda(), bf16(rng, pages, 4, 16, dim).cuda()
    q, kn, vn = bf16(rng, nodes, 24, dim).cuda(), bf16(rng, nodes, 4, dim).cuda(), bf16(rng, nodes, 4, dim).cuda()
    shape = native.Shape([0, nodes], pages, pages, num_q_heads=24, num_kv_heads=4, head_dim=dim)
    out16, status = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws16 = torch.empty(max(16, native.sd_verify_attn_workspace_size(shape)), dtype=torch.uint8, device="cuda")
    table, ctx, par = cu([range(pages)], torch.int32), cu([pages * 16 - 3], torch.int32), cu(chain(nodes), torch.int32)
    rot, pos = rope_table(1024, 64), cu(range(nodes), torch.int32)
    q_turned, k_turned = torch.empty_like(q), torch.empty_like(kn)
    logits = torch.randn(5, 20000, device="cuda")
    ids, best, entropy = torch.empty(5, 8, dtype=torch.int32, device="cuda"), torch.empty(5, 8, device="cuda"), torch.empty(5, device="cuda")
    lp_ws = torch.empty(native.sd_logprobs_workspace_size(5, 20000, 8), dtype=torch.uint8, device="cuda")
    cache = torch.zeros(1, *native.kv4_cache_shape(4, 4, dim), dtype=torch.uint8, device="cuda")
    slots = cu(range(16, 16 + nodes), torch.int32)
    calls = [
        lambda: native.sd_verify_attn(shape, q, kc, vc, kn, vn, table, ctx, par, out16, workspace=ws16, dev_status=status),
        lambda: wide.call(),
        lambda: native.sd_rope_append(rot, pos, q=q, k=kn, q_out=q_turned, k_out=k_turned, dev_status=status),
        lambda: small.call(),
        lambda: native.sd_kv4_append(cache, k_turned[None], vn[None], slots, dev_status=status),
        lambda: eight.call(),
        lambda: native.sd_logprobs(logits, None, None, ids, best, entropy, workspace=lp_ws, dev_status=status),
    ]
    outs = [out16, wide.out, q_turned, small.out, cache, eight.out, best]
    want = []
    for call, out in zip(calls, outs):
        call()
        torch.cuda.synchronize()
        want.append(out.clone())
    order = [0, 1, 3, 1, 0, 3, 2, 4, 1, 5, 3, 6, 0, 2, 5, 1, 6, 4, 3, 0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in order:
            calls[i]()
    for how in (lambda: [calls[i]() for i in order], graph.replay, graph.replay):
        for i, out in enumerate(outs):
            if i not in (2, 4):
                out.fill_(7)
        how()
        torch.cuda.synchronize()
        for i, (got, ref) in enumerate(zip(outs, want)):
            if i in (1, 3):
                got, ref = got[:-1], ref[:-1]
            if i == 5:
                got, ref = got[:eight.indptr[-1]], ref[:eight.indptr[-1]]
            assert torch.equal(got, ref), i
        assert int(status) == 0 and int(wide.status) == 0 and int(small.status) == 0
