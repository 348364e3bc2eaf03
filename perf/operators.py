"""The 8-bit block-scaled K/V cache operators, measured: page tables and slot maps, the quantising append, the attention.

``run`` computes each operator in its plain form with elementary torch operations, or, where ``own`` is true,
through the library's calls (``speculative_decoding_verify_decode_gb300.native``).  A cache page holds 16 tokens
of every KV head as e4m3 codes, and each (page, KV head) of K and of V has one fp32 scale: a code stands for
decode(code) * scale.
"""
import math
import random

import torch

own = False

PAGE = 16
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -100, 100     # the append's power-of-two scales are 2^MIN_EXP .. 2^MAX_EXP
DEVICE = "cuda"

# Head geometries (query heads, KV heads, head dim): the library's own, and a generic grouped-query one.
WIDE = (24, 4, 256)
NARROW = (32, 8, 128)


# ------------------------------------------------------------------------------------------ cases

def _attn(name, batch, nodes, tree, ctx_lo, ctx_hi, heads=WIDE, window=0, softcap=0.0, slopes=False, lens_seed=1):
    case = {"op": "attn", "batch": batch, "nodes": nodes, "tree": tree, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "hq": heads[0], "hkv": heads[1], "dim": heads[2], "window": window, "softcap": softcap,
            "slopes": slopes, "lens_seed": lens_seed}
    return dict(case, name=name) if name else case


def _append(name, layers, batch, rows_lo, rows_hi, ctx_hi, heads=WIDE, path=False, lens_seed=1):
    case = {"op": "append", "layers": layers, "batch": batch, "rows_lo": rows_lo, "rows_hi": rows_hi,
            "ctx_hi": ctx_hi, "hkv": heads[1], "dim": heads[2], "path": path, "lens_seed": lens_seed}
    return dict(case, name=name) if name else case


def _pages(name, op, batch, add_lo, add_hi, ctx_hi, path=False, lens_seed=1):
    case = {"op": op, "batch": batch, "add_lo": add_lo, "add_hi": add_hi, "ctx_hi": ctx_hi, "path": path,
            "lens_seed": lens_seed}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token of one short conversation: the smallest call, where latency counts
        _attn("attn_decode_ctx512", 1, 1, False, 512, 512),
        # a chain of eight drafts and its root at a few thousand tokens, the bench's short workload
        _attn("attn_chain9_ctx4k", 1, 9, False, 4096, 4096),
        # a draft tree of 22 nodes and its root, at the bench's two long contexts
        _attn("attn_tree23_ctx32k", 1, 23, True, 32768, 32768),
        _attn("attn_tree23_ctx128k", 1, 23, True, 131072, 131072),
        # eight streams with chains of four drafts and ragged contexts
        _attn("attn_chain5_b8_ragged", 8, 5, False, 1024, 16384, lens_seed=3),
        # single-token decoding of a large batch, contexts from one token up, the narrower heads
        _attn("attn_decode_b64_ragged", 64, 1, False, 1, 32768, heads=NARROW, lens_seed=5),
        # a target with capped scores and a distance bias, an odd context and an odd tree
        _attn("attn_tree31_capped_bias", 1, 31, True, 20001, 20001, heads=NARROW, softcap=50.0, slopes=True,
              lens_seed=7),
        # the accepted path of one step of sixteen layers
        _append("append_commit_16_layers", 16, 1, 6, 6, 4000, path=True),
        # a prompt's K/V of one layer, behind a context that ends inside a page
        _append("append_prompt_8191", 1, 1, 8191, 8191, 21, lens_seed=4),
        # the page tables and the slot map of a step's accepted paths
        _pages("extend_commit_b8", "extend", 8, 1, 9, 16384, path=True, lens_seed=2),
        # page tables and slot maps of a whole batch of prompts
        _pages("extend_prompts_b256", "extend", 256, 1, 32768, 5000, lens_seed=6),
        # the same batch rolled back to its prefixes: the pages return to the free list
        _pages("release_b256", "release", 256, 1, 32768, 5000, lens_seed=6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    seed = rng.randrange(1 << 20)
    kind = rng.choice(("attn", "attn", "append", "extend", "release"))
    if kind == "attn":
        heads = rng.choice((WIDE, NARROW))
        nodes = rng.choice((1, 1, _log_int(rng, 2, 64)))
        batch = _log_int(rng, 1, 128)
        most = min(131072, 1000000 // (batch * max(1, nodes // 3)))   # context tokens of a sequence
        hi = _log_int(rng, 1, max(2, most))
        lo = hi if batch == 1 else max(0, hi // rng.choice((1, 2, 1000000)))
        mods = rng.choice((0, 0, 1, 2, 3))
        window = rng.choice((0, 0, 0, _log_int(rng, 1, 8192)))
        return _attn("", batch, nodes, nodes > 2 and rng.random() < 0.6, min(lo, hi), hi, heads, window,
                     30.0 if mods & 1 else 0.0, bool(mods & 2), seed)
    if kind == "append":
        heads = rng.choice((WIDE, NARROW))
        layers = rng.choice((1, 1, _log_int(rng, 2, 32)))
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, 32768 // (batch * layers)))
        return _append("", layers, batch, rng.choice((0, 1, hi)) if batch > 1 else hi, hi, _log_int(rng, 1, 20000),
                       heads, hi <= 16 and rng.random() < 0.5, seed)
    batch = _log_int(rng, 1, 256)
    hi = _log_int(rng, 1, 32768)
    return _pages("", kind, batch, rng.choice((0, 1, hi)) if batch > 1 else hi, hi, _log_int(rng, 1, 32768),
                  kind == "extend" and hi <= 16 and rng.random() < 0.5, seed)


def _lens(case, lo, hi, salt):
    rng = random.Random(case["lens_seed"] * 7919 + salt)
    return [rng.randint(lo, hi) for _ in range(case["batch"])]


def _trees(case):
    """Parent ids of every sequence's draft nodes: chains, or trees whose node count varies over the batch."""
    rng = random.Random(case["lens_seed"] * 7919 + 2)
    out = []
    for b in range(case["batch"]):
        n = case["nodes"] if b == 0 or not case["tree"] else rng.randint(1, case["nodes"])
        out.append([-1] + [rng.randint(max(0, j - 4), j - 1) if case["tree"] else j - 1 for j in range(1, n)])
    return out


# ------------------------------------------------------------------------------------------ inputs

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _quantised(x):
    """Codes and power-of-two scales of [pages, heads, 16, dim] values, one scale per page and head."""
    amax = x.float().abs().amax(dim=(2, 3)).clamp(min=2.0 ** -60)
    scale = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)))
    codes = (x.float() / scale[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _cache(gen, pages, hkv, dim):
    """A cache as quantised keys or values leave it: normal values whose size differs from page to page and head to head."""
    codes = torch.empty(pages, hkv, PAGE, dim, dtype=torch.uint8, device=DEVICE)
    scales = torch.empty(pages, hkv, dtype=torch.float32, device=DEVICE)
    step = max(1, (1 << 27) // (hkv * PAGE * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, hkv, PAGE, dim, dtype=torch.bfloat16, device=DEVICE, generator=gen)
        size = torch.exp2(torch.rand(n, hkv, 1, 1, device=DEVICE, generator=gen) * 2 - 1)
        codes[p:p + n], scales[p:p + n] = _quantised(x * size)
    return codes, scales


def _table(gen, lens, extra):
    """A pool's page ids in random order, dealt to the sequences; entries past a sequence's pages are -1."""
    counts = [-(-n // PAGE) for n in lens]
    pool = sum(counts) + extra
    perm = torch.randperm(pool, device=DEVICE, generator=gen).to(torch.int32)
    width = max(1, max(counts))
    c = torch.tensor(counts, device=DEVICE)
    j = torch.arange(width, device=DEVICE)[None]
    first = (torch.cumsum(c, 0) - c)[:, None]
    table = torch.where(j < c[:, None], perm[(first + j).clamp(max=pool - 1)], -1).to(torch.int32).contiguous()
    return table, perm[sum(counts):], pool


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "attn":
        hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
        lens, trees = _lens(case, case["ctx_lo"], case["ctx_hi"], 1), _trees(case)
        indptr = [0]
        for t in trees:
            indptr.append(indptr[-1] + len(t))
        s["table"], _, pool = _table(gen, lens, 3)
        s["k"], s["ks"] = _cache(gen, pool, hkv, dim)
        s["v"], s["vs"] = _cache(gen, pool, hkv, dim)
        rand = lambda *shape: torch.randn(*shape, dtype=torch.bfloat16, device=DEVICE, generator=gen)  # noqa: E731
        s["q"], s["k_new"], s["v_new"] = (rand(indptr[-1], h, dim) for h in (hq, hkv, hkv))
        s["ctx"], s["parents"], s["indptr"] = _ints(lens), _ints(sum(trees, [])), indptr
        s["out"] = torch.empty_like(s["q"])
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEVICE) / hq) if case["slopes"] else None
        if own:
            from speculative_decoding_verify_decode_gb300 import native
            s["shape"] = native.Shape(indptr, s["table"].shape[1], pool, window=case["window"], num_q_heads=hq,
                                      num_kv_heads=hkv, head_dim=dim)
            s["ws"] = torch.empty(native.sd_kv8_attn_workspace_size(s["shape"]), dtype=torch.uint8, device=DEVICE)
        return s
    add = "rows" if case["op"] == "append" else "add"
    ctx, add = _lens(case, 0, case["ctx_hi"], 1), _lens(case, case[add + "_lo"], case[add + "_hi"], 3)
    grown = [c + a for c, a in zip(ctx, add)]
    table, free, pool = _table(gen, grown if case["op"] != "extend" else ctx, 3)
    if case["op"] == "append":
        layers, hkv, dim, total = case["layers"], case["hkv"], case["dim"], max(1, sum(add))
        b = torch.repeat_interleave(torch.arange(len(add), device=DEVICE), torch.tensor(add, device=DEVICE))
        i = torch.arange(sum(add), device=DEVICE) - (torch.cumsum(_ints(add), 0) - _ints(add))[b]
        pos = _ints(ctx)[b] + i
        s["slots"] = torch.full((total + 5,), -1, dtype=torch.int32, device=DEVICE)   # room behind the last row
        s["slots"][:sum(add)] = table[b, pos // PAGE] * PAGE + (pos % PAGE).to(torch.int32)
        source = total if not case["path"] else 3 * total
        s["rows"] = None
        if case["path"]:       # the accepted nodes among three times as many
            s["rows"] = torch.zeros(total + 5, dtype=torch.int32, device=DEVICE)
            s["rows"][:total] = torch.sort(torch.randperm(source, device=DEVICE, generator=gen)[:total])[0]
        caches = [[_cache(gen, pool, hkv, dim) for _ in range(layers)] for _ in "kv"]
        s["k"], s["v"] = (torch.stack([c for c, _ in x]) for x in caches)
        s["ks"], s["vs"] = (torch.stack([c for _, c in x]) for x in caches)
        size = torch.exp2(torch.rand(source, hkv, 1, device=DEVICE, generator=gen) * 4 - 2)
        new = lambda: (torch.randn(layers, source, hkv, dim, device=DEVICE, generator=gen) * size).bfloat16()  # noqa: E731
        s["k_new"], s["v_new"] = new(), new()
        return s
    # page tables: the pool keeps room for every sequence at its largest
    batch = len(ctx)
    width = max(1, max(-(-n // PAGE) for n in grown))
    held = [-(-n // PAGE) for n in (ctx if case["op"] == "extend" else grown)]
    pool = sum(-(-n // PAGE) for n in grown) + 7
    perm = torch.randperm(pool, device=DEVICE, generator=gen).to(torch.int32)
    h = torch.tensor(held, device=DEVICE)
    j = torch.arange(width, device=DEVICE)[None]
    at = (torch.cumsum(h, 0) - h)[:, None] + j
    s["table"] = torch.where(j < h[:, None], perm[at.clamp(max=pool - 1)], -1).to(torch.int32).contiguous()
    used = sum(held)
    s["free_list"] = torch.cat([perm[used:], torch.full((used,), -1, dtype=torch.int32, device=DEVICE)])
    s["free_count"], s["held"], s["ctx"], s["add"] = _ints([pool - used]), _ints(held), _ints(ctx), _ints(add)
    s["new_free_count"], s["new_held"] = torch.empty_like(s["free_count"]), torch.empty_like(s["held"])
    s["q_indptr"] = s["path"] = s["rows"] = None
    if case["op"] == "extend":
        s["slots"] = torch.empty(sum(add) + 3, dtype=torch.int32, device=DEVICE)      # room for a few rows more
        s["row_indptr"] = torch.empty(batch + 1, dtype=torch.int32, device=DEVICE)
        s["new_ctx"] = torch.empty_like(s["ctx"])
        if case["path"]:
            nodes = 3 * max(1, case["add_hi"])
            s["q_indptr"] = list(range(0, (batch + 1) * nodes, nodes))
            order = torch.rand(batch, nodes, device=DEVICE, generator=gen).argsort(dim=1)[:, :max(1, case["add_hi"])]
            s["path"] = torch.sort(order, dim=1)[0].to(torch.int32).contiguous()
            s["starts"] = _ints(s["q_indptr"])
            s["rows"] = torch.empty_like(s["slots"])
    return s


# ------------------------------------------------------------------------------------------ the calls

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    return {"attn": _plain_attn, "append": _plain_append, "extend": _plain_extend, "release": _plain_release}[case["op"]](s, case)


def _run_own(s, case):
    from speculative_decoding_verify_decode_gb300 import native
    if case["op"] == "attn":
        native.sd_kv8_attn(s["shape"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["k_new"], s["v_new"], s["table"],
                           s["ctx"], s["parents"], s["out"], softcap=case["softcap"], slopes=s["slopes"],
                           workspace=s["ws"])
        return s["out"]
    if case["op"] == "append":
        native.sd_kv8_append(s["k"], s["v"], s["ks"], s["vs"], s["k_new"], s["v_new"], s["slots"], s["rows"])
        return _cache_values(s["k"], s["v"], s["ks"], s["vs"])
    if case["op"] == "extend":
        native.sd_pages_extend(s["ctx"], s["add"], s["table"], s["held"], s["new_held"], s["free_list"],
                               s["free_count"], s["new_free_count"], s["slots"], rows=s["rows"],
                               row_indptr=s["row_indptr"], new_ctx_lens=s["new_ctx"], q_indptr=s["q_indptr"],
                               path=s["path"])
        return (s["table"], s["new_held"], s["new_free_count"], s["slots"], s["row_indptr"], s["new_ctx"], s["rows"])
    native.sd_pages_release(s["ctx"], s["table"], s["held"], s["new_held"], s["free_list"], s["free_count"],
                            s["new_free_count"])
    return s["new_held"], s["free_list"], s["new_free_count"]


def _cache_values(k, v, ks, vs):
    return k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs


# ------------------------------------------------------------------------------------------ plain forms

def _decoded(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * scales[..., None, None]


def _plain_attn(s, case):
    """Scores of all keys at once, masked; a softmax written out; the weighted sum."""
    q, ctx, indptr = s["q"].float(), s["ctx"].long(), torch.tensor(s["indptr"], device=DEVICE)
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    batch, nmax = len(s["indptr"]) - 1, max(b - a for a, b in zip(s["indptr"], s["indptr"][1:]))
    counts = indptr[1:] - indptr[:-1]
    j = torch.arange(nmax, device=DEVICE)
    at = (indptr[:-1, None] + j).clamp(max=q.shape[0] - 1)            # rows padded to [batch, nmax]
    is_node = j < counts[:, None]
    # the draft block's masks: each node sees its root path
    par = torch.where(is_node, s["parents"].long()[at], -1)
    seen = torch.eye(nmax, device=DEVICE) + (par[:, :, None] == j).float()
    for _ in range(max(1, math.ceil(math.log2(nmax)))):
        seen = (seen @ seen > 0).float()
    depth = seen.sum(-1).long() - 1
    # keys: context pages, then the draft block
    table = s["table"].long().clamp(min=0)
    held = lambda c, sc: _decoded(c[table], sc[table]).transpose(1, 2).reshape(batch, hkv, -1, dim)  # noqa: E731
    block = lambda x: x.float()[at].transpose(1, 2)                   # noqa: E731
    pos = torch.arange(table.shape[1] * PAGE, device=DEVICE)
    q_pos = ctx[:, None] + depth                                       # [batch, nmax]
    k_pos = torch.cat([pos.expand(batch, -1), q_pos], 1)
    cached = pos < ctx[:, None]
    mask = torch.cat([cached[:, None, :].expand(-1, nmax, -1), (seen > 0) & is_node[:, None, :]], 2)
    if case["window"]:
        mask = mask & (k_pos[:, None, :] > q_pos[:, :, None] - case["window"])
    rows = q[at].reshape(batch, nmax, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, dim)
    k = torch.cat([held(s["k"], s["ks"]), block(s["k_new"])], 2)
    score = (rows @ k.transpose(2, 3)).reshape(batch, hkv, hq // hkv, nmax, -1) / math.sqrt(dim)
    del k
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    if s["slopes"] is not None:
        away = (k_pos[:, None, :] - q_pos[:, :, None]).float()
        score = score + s["slopes"].reshape(hkv, hq // hkv, 1, 1) * away[:, None, None]
    score = torch.where(mask[:, None, None], score, float("-inf"))
    w = torch.exp(score - score.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    v = held(s["v"], s["vs"]).masked_fill(~cached[:, None, :, None], 0.0)
    v = torch.cat([v, block(s["v_new"])], 2)
    out = w.reshape(batch, hkv, -1, w.shape[-1]) @ v
    out = out.reshape(batch, hkv, hq // hkv, nmax, dim).permute(0, 3, 1, 2, 4).reshape(batch, nmax, hq, dim)
    return out[is_node].bfloat16()


def _plain_append(s, case):
    """Amax of each touched page and head, its scale, the old codes on the new scale, the new codes; in place."""
    live = s["slots"] >= 0
    slots = s["slots"].long()[live]
    src = s["rows"].long()[live] if s["rows"] is not None else torch.arange(s["slots"].numel(), device=DEVICE)[live]
    pages, at = torch.unique(slots // PAGE, return_inverse=True)
    off = slots % PAGE
    first = torch.full_like(pages, PAGE).scatter_reduce(0, at, off, "amin")               # the first new token of a page
    old = torch.arange(PAGE, device=DEVICE) < first[:, None]                              # [pages, 16]
    for c in "kv":
        x, codes, scales = s[c + "_new"][:, src].float(), s[c][:, pages], s[c + "s"][:, pages]
        finite = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)                    # [layers, rows, heads]
        amax = torch.zeros_like(scales).scatter_reduce(1, at[None, :, None].expand_as(finite), finite, "amax")
        # the smallest 2^e with amax <= 448 * 2^e; frexp gives amax = m * 2^e with m in [1/2, 1), and 448 = 0.875 * 2^9
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), MIN_EXP).clamp(MIN_EXP, MAX_EXP)
        need = torch.ldexp(torch.ones_like(amax), e)
        scale = torch.where((first > 0)[None, :, None], torch.maximum(scales, need), need)
        moved = (_decoded(codes, scales) / scale[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX)
        codes = torch.where(old[None, :, None, :, None], moved.to(torch.float8_e4m3fn).view(torch.uint8), codes)
        rows = (x / scale[:, at][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        codes[:, at, :, off] = rows.view(torch.uint8).transpose(0, 1)
        s[c][:, pages], s[c + "s"][:, pages] = codes, scale
    return _cache_values(s["k"], s["v"], s["ks"], s["vs"])


def _plain_extend(s, case):
    ctx, add, held, count = s["ctx"].long(), s["add"].long(), s["held"].long(), s["free_count"].long()
    need = torch.maximum(held, (ctx + add + PAGE - 1) // PAGE)
    grow = need - held
    first = torch.cumsum(grow, 0) - grow
    j = torch.arange(s["table"].shape[1], device=DEVICE)[None]
    fresh = (j >= held[:, None]) & (j < need[:, None])
    take = (count - 1 - (first[:, None] + j - held[:, None])).clamp(0, s["free_list"].numel() - 1)
    table = torch.where(fresh, s["free_list"][take], s["table"])
    ends = torch.cumsum(add, 0)
    r = torch.arange(s["slots"].numel(), device=DEVICE)
    b = torch.searchsorted(ends, r, right=True).clamp(max=ctx.numel() - 1)
    i = r - (ends - add)[b]
    live = r < ends[-1]
    pos = torch.where(live, ctx[b] + i, 0)
    slots = torch.where(live, table[b, pos // PAGE].long() * PAGE + pos % PAGE, -1).int()
    rows = None
    if s["path"] is not None:
        rows = torch.where(live, s["starts"][b] + s["path"][b, torch.where(live, i, 0)], -1).int()
    indptr = torch.cat([torch.zeros_like(ends[:1]), ends]).int()
    return table, need.int(), (count - grow.sum()).int(), slots, indptr, (ctx + add).int(), rows


def _plain_release(s, case):
    keep, held, count = (s["ctx"].long() + PAGE - 1) // PAGE, s["held"].long(), s["free_count"].long()
    left = torch.minimum(keep, held)
    gone = held - left
    j = torch.arange(s["table"].shape[1], device=DEVICE)[None]
    back = (j >= left[:, None]) & (j < held[:, None])
    pages = s["table"][back]                                           # by sequence, then by position
    n = s["free_list"].numel()
    at = torch.arange(n, device=DEVICE) - count
    total = gone.sum()
    padded = torch.cat([pages, pages.new_zeros(n)])
    free = torch.where((at >= 0) & (at < total), padded[at.clamp(min=0)], s["free_list"])
    return left.int(), free, (count + total).int()


# ------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s, case)
    if case["op"] == "append":
        return _exact_append(s, case)
    return None        # whole numbers


def _e4m3_values():
    """Value of each of the 256 codes: sign, four exponent bits with bias 7, three mantissa bits."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = math.nan if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-a if c & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=DEVICE)


def _exact_attn(s, case):
    """One sequence, one KV head at a time; the scores of each node over its own keys."""
    value = _e4m3_values()
    group, parents = case["hq"] // case["hkv"], s["parents"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(s["ctx"].tolist()):
        lo, hi = s["indptr"][b], s["indptr"][b + 1]
        paths = []
        for i in range(hi - lo):
            up = parents[lo + i]
            paths.append((paths[up] if up >= 0 else []) + [i])
        depth = torch.tensor([len(p) - 1 for p in paths], device=DEVICE)
        see = torch.zeros(hi - lo, n + hi - lo, dtype=torch.bool, device=DEVICE)
        see[:, :n] = True
        for i, p in enumerate(paths):
            see[i, [n + x for x in p]] = True
        key_at = torch.cat([torch.arange(n, device=DEVICE), n + depth])
        away = key_at[None, :] - (n + depth)[:, None]
        if case["window"]:
            see &= away > -case["window"]
        pages = s["table"][b, :-(-n // PAGE)].long()
        for g in range(case["hkv"]):
            def keys(codes, scales, new):
                x = value[codes[pages, g].long()] * scales[pages, g].double()[:, None, None]
                return torch.cat([x.reshape(-1, case["dim"])[:n], new[lo:hi, g].double()])
            q = s["q"][lo:hi, g * group:(g + 1) * group].double()
            t = torch.einsum("nhd,kd->hnk", q, keys(s["k"], s["ks"], s["k_new"])) * case["dim"] ** -0.5
            if case["softcap"]:
                t = torch.tanh(t / case["softcap"]) * case["softcap"]
            if s["slopes"] is not None:
                t += s["slopes"][g * group:(g + 1) * group].double()[:, None, None] * away
            t = torch.softmax(t.masked_fill(~see, -math.inf), -1)
            out[lo:hi, g * group:(g + 1) * group] = torch.einsum("hnk,kd->nhd", t, keys(s["v"], s["vs"], s["v_new"]))
    return out


def _exact_append(s, case):
    """Page by page, as a sequence's rows arrive; every code the nearest value of the format, ties to the even code."""
    value = _e4m3_values()
    finite = value[:127]                                               # 0 .. 448, rising
    mids = (finite[1:] + finite[:-1]) / 2

    def nearest(x):
        a = x.abs()
        up, down = torch.searchsorted(mids, a, right=True), torch.searchsorted(mids, a, right=False)
        code = torch.where((up != down) & (down % 2 == 0), down, up)   # on a midpoint the even code of the two
        return torch.where(torch.signbit(x), -finite[code], finite[code])

    slots = s["slots"].tolist()
    rows = s["rows"].tolist() if s["rows"] is not None else list(range(len(slots)))
    groups = {}
    for slot, row in zip(slots, rows):
        if slot >= 0:
            groups.setdefault(slot // PAGE, []).append((slot % PAGE, row))
    out = []
    for c in "kv":
        codes, scales, new = s[c], s[c + "s"].double(), s[c + "_new"].double()
        got = value[codes.long()] if codes.numel() < 1 << 29 else None
        if got is None:
            return None
        for page, items in groups.items():
            first = min(o for o, _ in items)
            x = new[:, [r for _, r in items]]                          # [layers, rows, heads, dim]
            amax = x.abs().amax(dim=(1, 3))
            scale = torch.exp2(torch.floor(torch.log2(amax / E4M3_MAX)) - 1)   # below the answer, by up to two steps
            for _ in range(3):
                scale = torch.where(amax <= E4M3_MAX * scale, scale, 2 * scale)
            if first:
                scale = torch.maximum(scale, scales[:, page])
                old = got[:, page, :, :first]
                got[:, page, :, :first] = nearest(old * (scales[:, page] / scale)[:, :, None, None])
            scales[:, page] = scale
            got[:, page, :, [o for o, _ in items]] = nearest(x / scale[:, None, :, None]).transpose(1, 2)
        out.append((got, scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]


# ------------------------------------------------------------------------------------------ the work of a pass

def work(case):
    if case["op"] == "attn":
        lens, nodes = _lens(case, case["ctx_lo"], case["ctx_hi"], 1), [len(t) for t in _trees(case)]
        spans = [min(n, case["window"] - 1) if case["window"] else n for n in lens]
        row = case["hkv"] * case["dim"]
        total, pages = sum(nodes), sum(-(-n // PAGE) for n in spans)
        size = sum(spans) * 2 * row + pages * (8 * case["hkv"] + 4) + total * (4 * case["hq"] * case["dim"] + 4 * row)
        flops = sum(4 * n * case["hq"] * case["dim"] * (span + 1) for n, span in zip(nodes, spans))
        return {"bytes": size, "flops": flops}
    if case["op"] == "append":
        add, ctx = _lens(case, case["rows_lo"], case["rows_hi"], 3), _lens(case, 0, case["ctx_hi"], 1)
        row = case["hkv"] * case["dim"]
        old = sum(c % PAGE for c, a in zip(ctx, add) if a)
        values = case["layers"] * 2 * row * (3 * sum(add) + old)
        return {"bytes": values + 4 * (sum(add) + 5), "flops": 2 * case["layers"] * 2 * row * sum(add)}
    ctx, add = _lens(case, 0, case["ctx_hi"], 1), _lens(case, case["add_lo"], case["add_hi"], 3)
    fresh = sum(-(-(c + a) // PAGE) - -(-c // PAGE) for c, a in zip(ctx, add))
    rows = sum(add) * (12 if case["path"] else 4) if case["op"] == "extend" else 0
    return {"bytes": 24 * case["batch"] + 8 * fresh + rows, "flops": 0}
