"""The 4-bit K/V cache's operators, the rotating append and the log probabilities, measured.

``run`` computes each operator in its plain form with elementary torch operations, or, where ``own`` is true,
through the library's calls (``speculative_decoding_verify_decode_gb300.native``).

A page of the 4-bit cache holds 16 tokens of every KV head; a value is (c - 8) * s with a 4-bit code c and a scale s
of its token and 32 dims (bf16 with 5 significant bits).  One (page, KV head) of a cache uint8
[pages, heads, 2, 9 * dim] is a K record and a V record of 9 * dim bytes each:
  K  codes [dim / 32][16 tokens][16 bytes: 32 dims], then scales bf16 [16 tokens][dim / 32]
  V  codes [dim][8 bytes: 16 tokens], then scales bf16 [dim / 32][16 tokens]
Eight codes make a little-endian word, code e at bit 16 * (e % 2) + 4 * (e // 2).
"""
import math
import random

import torch

own = False

PAGE, BLOCK = 16, 32
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


def _rows(name, op, layers, batch, rows_lo, rows_hi, ctx_hi, heads=WIDE, path=False, lens_seed=1):
    """Rows of every sequence into the 4-bit cache ("append"), or back out of it ("read")."""
    case = {"op": op, "layers": layers, "batch": batch, "rows_lo": rows_lo, "rows_hi": rows_hi, "ctx_hi": ctx_hi,
            "hkv": heads[1], "dim": heads[2], "path": path, "lens_seed": lens_seed}
    return dict(case, name=name) if name else case


def _rope(name, batch, rows_lo, rows_hi, ctx_hi, heads=WIDE, rot=256, interleaved=False, cache=True, lens_seed=1):
    case = {"op": "rope", "batch": batch, "rows_lo": rows_lo, "rows_hi": rows_hi, "ctx_hi": ctx_hi, "hq": heads[0],
            "hkv": heads[1], "dim": heads[2], "rot": rot, "interleaved": interleaved, "cache": cache,
            "lens_seed": lens_seed}
    return dict(case, name=name) if name else case


def _logprobs(name, rows, vocab, dtype, given, top, temperature=1.0):
    case = {"op": "logprobs", "rows": rows, "vocab": vocab, "dtype": dtype, "given": given, "top": top,
            "temperature": temperature}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token of one short conversation: the smallest call, where latency counts
        _attn("attn_decode_ctx512", 1, 1, False, 512, 512),
        # a draft tree of 22 nodes and its root over the bench's longest context
        _attn("attn_tree23_ctx128k", 1, 23, True, 131072, 131072),
        # single-token decoding of a large batch, contexts from one token up, the narrower heads
        _attn("attn_decode_b64_ragged", 64, 1, False, 1, 32768, heads=NARROW, lens_seed=5),
        # a target with capped scores and a distance bias, an odd context and an odd tree
        _attn("attn_tree31_capped_bias", 1, 31, True, 20001, 20001, heads=NARROW, softcap=50.0, slopes=True,
              lens_seed=7),
        # the accepted path of one step of sixteen layers
        _rows("append_commit_16_layers", "append", 16, 1, 6, 6, 4000, path=True),
        # a prompt's K/V of one layer, behind a context that ends inside a page
        _rows("append_prompt_8191", "append", 1, 1, 8191, 8191, 21, lens_seed=4),
        # a long sequence of one layer taken out of the cache, to be held elsewhere
        _rows("read_16383", "read", 1, 1, 16383, 16383, 1, lens_seed=3),
        # the last tokens of eight streams, every layer's
        _rows("read_tails_b8", "read", 16, 8, 16, 16, 4000, lens_seed=9),
        # the draft blocks of eight streams rotated before a verify step
        _rope("rope_drafts_b8", 8, 5, 5, 16384, cache=False, lens_seed=2),
        # a prompt rotated and appended, a quarter of each head rotating, at far positions
        _rope("rope_prompt_8191", 1, 8191, 8191, 100000, rot=64, lens_seed=4),
        # what a server returns beside the tokens of one tree verify
        _logprobs("logprobs_tree23", 23, 151936, "float32", 1, 5),
        # the log probabilities of a prompt's own tokens, twenty alternatives each
        _logprobs("logprobs_prompt_2047", 2047, 151936, "bfloat16", 1, 20, 0.7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    seed = rng.randrange(1 << 20)
    kind = rng.choice(("attn", "attn", "append", "read", "rope", "logprobs"))
    heads = rng.choice((WIDE, NARROW))
    if kind == "attn":
        nodes = rng.choice((1, 1, _log_int(rng, 2, 64)))
        batch = _log_int(rng, 1, 128)
        most = min(131072, 1000000 // (batch * max(1, nodes // 3)))   # context tokens of a sequence
        hi = _log_int(rng, 1, max(2, most))
        lo = hi if batch == 1 else max(0, hi // rng.choice((1, 2, 1000000)))
        mods = rng.choice((0, 0, 1, 2, 3))
        window = rng.choice((0, 0, 0, _log_int(rng, 1, 8192)))
        return _attn("", batch, nodes, nodes > 2 and rng.random() < 0.6, min(lo, hi), hi, heads, window,
                     30.0 if mods & 1 else 0.0, bool(mods & 2), seed)
    if kind in ("append", "read"):
        layers = rng.choice((1, 1, _log_int(rng, 2, 32)))
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, 32768 // (batch * layers)))
        return _rows("", kind, layers, batch, rng.choice((0, 1, hi)) if batch > 1 else hi, hi, _log_int(rng, 1, 20000),
                     heads, kind == "append" and hi <= 16 and rng.random() < 0.5, seed)
    if kind == "rope":
        batch = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(1, 16384 // batch))
        rot = rng.choice((heads[2], heads[2], heads[2] // 2, heads[2] // 4, 48))
        return _rope("", batch, rng.choice((1, hi)), hi, _log_int(rng, 1, 131072), heads, rot, rng.random() < 0.3,
                     rng.random() < 0.6, seed)
    vocab = rng.choice((151936, 32000, 50257, _log_int(rng, 64, 200000)))
    rows = _log_int(rng, 1, max(1, min(4096, 300000000 // vocab)))
    return _logprobs("", rows, vocab, rng.choice(("float32", "bfloat16", "float16")), rng.choice((0, 1, 1, 4)),
                     rng.choice((0, 1, 5, 20, 32)), rng.choice((1.0, 1.0, 0.6, 1.3)))


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


# ------------------------------------------------------------------------------------------ the 4-bit format

def _codes_and_scales(x):
    """x [..., dim] fp32 -> codes 0..15 (int32, same shape) and scales bf16 [..., dim / 32].

    A block's scale is its value largest in magnitude (the first of them) divided by -8, rounded to 5 significant bits
    (ties to even); blocks below 2^-100 have scale 0 and codes 8."""
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.gather(-1, b.abs().argmax(-1, keepdim=True))[..., 0]
    m, e = torch.frexp(top / -8)                                  # 0.5 <= |m| < 1
    s = torch.ldexp(torch.round(m * 32), e - 5)                   # 5 bits, ties to even
    s = torch.where(top.abs() < 2.0 ** -100, 0.0, s)
    c = torch.round(b / torch.where(s == 0, 1.0, s)[..., None]) + 8
    c = torch.where(s[..., None] == 0, 8.0, c.clamp(0, 15))
    return c.int().flatten(-2), s.bfloat16()


def _words(c):
    """Codes [..., 8 n] -> little-endian words as bytes [..., 4 n]."""
    c = c.unflatten(-1, (-1, 8)).to(torch.int64)
    shift = torch.tensor([16 * (e % 2) + 4 * (e // 2) for e in range(8)], device=c.device)
    w = (c << shift).sum(-1)
    return torch.stack([(w >> (8 * i)) & 255 for i in range(4)], -1).to(torch.uint8).flatten(-2)


def _unwords(b):
    """The reverse: bytes [..., 4 n] -> codes [..., 8 n] (int32)."""
    b = b.unflatten(-1, (-1, 4)).to(torch.int32)
    w16 = torch.stack([b[..., 0] | b[..., 1] << 8, b[..., 2] | b[..., 3] << 8], -1)   # codes 0 2 4 6, codes 1 3 5 7
    shift = torch.arange(0, 16, 4, device=b.device, dtype=torch.int32)
    return ((w16[..., None, :] >> shift[:, None]) & 15).flatten(-3)


def _pages_of(k, v):
    """Values [pages, heads, 16, dim] -> cache pages uint8 [pages, heads, 2, 9 dim]."""
    n, h, _, dim = k.shape
    ck, sk = _codes_and_scales(k)
    cv, sv = _codes_and_scales(v)
    kb = _words(ck).reshape(n, h, PAGE, dim // BLOCK, 16).transpose(2, 3).reshape(n, h, -1)
    vb = _words(cv.transpose(2, 3)).reshape(n, h, -1)
    raw = lambda s: s.contiguous().view(torch.uint8).reshape(n, h, -1)  # noqa: E731
    return torch.stack([torch.cat([kb, raw(sk)], -1), torch.cat([vb, raw(sv.transpose(2, 3))], -1)], 2)


def _values(pages, dim):
    """Cache pages [..., 2, 9 dim] -> K and V values fp32 [..., 16, dim]."""
    nb, cut = dim // BLOCK, 8 * dim
    lead = pages.shape[:-2]
    k, v = pages[..., 0, :], pages[..., 1, :]
    scales = lambda r: r[..., cut:].contiguous().view(torch.bfloat16).float()  # noqa: E731
    sk, sv = scales(k).reshape(*lead, PAGE, nb), scales(v).reshape(*lead, nb, PAGE).transpose(-1, -2)
    ck = _unwords(k[..., :cut].reshape(*lead, nb, PAGE, 16).transpose(-2, -3).reshape(*lead, PAGE, dim // 2))
    cv = _unwords(v[..., :cut].reshape(*lead, dim, 8)).transpose(-1, -2)
    spread = lambda s: s.repeat_interleave(BLOCK, -1)  # noqa: E731
    return (ck - 8) * spread(sk), (cv - 8) * spread(sv)


# ------------------------------------------------------------------------------------------ inputs

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _cache(gen, pages, hkv, dim):
    """A cache as quantised keys and values leave it: normal values whose size differs from page to page and head to head."""
    out = torch.empty(pages, hkv, 2, 9 * dim, dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (hkv * PAGE * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        new = lambda: torch.randn(n, hkv, PAGE, dim, device=DEVICE, generator=gen) * torch.exp2(  # noqa: E731
            torch.rand(n, hkv, 1, 1, device=DEVICE, generator=gen) * 2 - 1)
        out[p:p + n] = _pages_of(new(), new())
    return out


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
    return table, pool


def _slot_map(table, ctx, add):
    """Positions and slots of the rows that join every sequence, in sequence order."""
    a, c = torch.tensor(add, device=DEVICE), torch.tensor(ctx, device=DEVICE)
    b = torch.repeat_interleave(torch.arange(len(add), device=DEVICE), a)
    pos = c[b] + torch.arange(sum(add), device=DEVICE) - (torch.cumsum(a, 0) - a)[b]
    return pos.int(), table[b, pos // PAGE] * PAGE + (pos % PAGE).int()


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, dtype=torch.bfloat16, device=DEVICE, generator=gen)  # noqa: E731
    s = {"case": case}
    if case["op"] == "logprobs":
        rows, vocab, dtype = case["rows"], case["vocab"], getattr(torch, case["dtype"])
        # logits as a model gives them: a broad background, and one to three tokens well above it
        x = torch.empty(rows, vocab, dtype=dtype, device=DEVICE)
        for r in range(0, rows, 256):
            x[r:r + 256] = torch.randn(min(256, rows - r), vocab, device=DEVICE, generator=gen) * 2.5
        peaks = torch.randint(vocab, (rows, 3), device=DEVICE, generator=gen)
        up = torch.rand(rows, 3, device=DEVICE, generator=gen) * 20
        x.scatter_(1, peaks, up.to(dtype))
        s["logits"], s["given"] = x, None
        if case["given"]:      # the likely token, and others
            others = torch.randint(vocab, (rows, case["given"]), device=DEVICE, generator=gen)
            s["given"] = torch.cat([peaks[:, :1], others[:, 1:]], 1).to(torch.int32).contiguous()
        f32 = lambda *shape: torch.empty(*shape, device=DEVICE)  # noqa: E731
        s["lp"] = f32(rows, case["given"]) if case["given"] else None
        s["ids"] = torch.empty(rows, case["top"], dtype=torch.int32, device=DEVICE) if case["top"] else None
        s["top_lp"] = f32(rows, case["top"]) if case["top"] else None
        s["entropy"], s["lse"] = f32(rows), f32(rows)
        if own:
            from speculative_decoding_verify_decode_gb300 import native
            n = native.sd_logprobs_workspace_size(rows, vocab, case["top"])
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEVICE)
        return s
    if case["op"] == "attn":
        hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
        lens, trees = _lens(case, case["ctx_lo"], case["ctx_hi"], 1), _trees(case)
        indptr = [0]
        for t in trees:
            indptr.append(indptr[-1] + len(t))
        s["table"], pool = _table(gen, lens, 3)
        s["cache"] = _cache(gen, pool, hkv, dim)
        s["q"], s["k_new"], s["v_new"] = (rand(indptr[-1], h, dim) for h in (hq, hkv, hkv))
        s["ctx"], s["parents"], s["indptr"] = _ints(lens), _ints(sum(trees, [])), indptr
        s["out"] = torch.empty_like(s["q"])
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEVICE) / hq) if case["slopes"] else None
        if own:
            from speculative_decoding_verify_decode_gb300 import native
            s["shape"] = native.Shape(indptr, s["table"].shape[1], pool, window=case["window"], num_q_heads=hq,
                                      num_kv_heads=hkv, head_dim=dim)
            s["ws"] = torch.empty(native.sd_kv4_attn_workspace_size(s["shape"]), dtype=torch.uint8, device=DEVICE)
        return s
    ctx, add = _lens(case, 0, case["ctx_hi"] - 1, 1), _lens(case, case["rows_lo"], case["rows_hi"], 3)
    table, pool = _table(gen, [c + a for c, a in zip(ctx, add)], 3)
    pos, slots = _slot_map(table, ctx, add)
    total, hkv, dim = sum(add), case["hkv"], case["dim"]
    if case["op"] == "rope":
        hq, rot = case["hq"], case["rot"]
        qkv = rand(total, (hq + 2 * hkv) * dim)                   # the fused projection's rows
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, dim)) for x in qkv.split((hq * dim, hkv * dim, hkv * dim), 1))
        freq = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
        angle = torch.arange(max(c + a for c, a in zip(ctx, add)) + 1, device=DEVICE).double()[:, None] * freq
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["pos"], s["slots"] = pos, slots
        s["q_out"], s["k_out"] = (torch.empty(total, h, dim, dtype=torch.bfloat16, device=DEVICE) for h in (hq, hkv))
        if case["cache"]:
            s["k_cache"], s["v_cache"] = (rand(pool, hkv, PAGE, dim) for _ in "kv")
        return s
    layers = case["layers"]
    s["slots"] = torch.full((total + 5,), -1, dtype=torch.int32, device=DEVICE)   # room behind the last row
    s["slots"][:total] = slots
    s["cache"] = torch.stack([_cache(gen, pool, hkv, dim) for _ in range(layers)])
    s["k_out"], s["v_out"] = (torch.zeros(layers, total + 5, hkv, dim, dtype=torch.bfloat16, device=DEVICE) for _ in "kv")
    if case["op"] == "append":
        source = max(1, total) if not case["path"] else 3 * total
        s["rows"] = None
        if case["path"]:       # the accepted nodes among three times as many
            s["rows"] = torch.zeros(total + 5, dtype=torch.int32, device=DEVICE)
            s["rows"][:total] = torch.sort(torch.randperm(source, device=DEVICE, generator=gen)[:total])[0]
        size = torch.exp2(torch.rand(source, hkv, 1, device=DEVICE, generator=gen) * 4 - 2)
        new = lambda: (torch.randn(layers, source, hkv, dim, device=DEVICE, generator=gen) * size).bfloat16()  # noqa: E731
        s["k_new"], s["v_new"] = new(), new()
    return s


# ------------------------------------------------------------------------------------------ the calls

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    return {"attn": _plain_attn, "append": _plain_append, "read": _plain_read, "rope": _plain_rope,
            "logprobs": _plain_logprobs}[case["op"]](s, case)


def _run_own(s, case):
    from speculative_decoding_verify_decode_gb300 import native
    if case["op"] == "attn":
        native.sd_kv4_attn(s["shape"], s["q"], s["cache"], s["k_new"], s["v_new"], s["table"], s["ctx"], s["parents"],
                           s["out"], softcap=case["softcap"], slopes=s["slopes"], workspace=s["ws"])
        return s["out"]
    if case["op"] == "append":     # and what the cache then holds for these rows
        native.sd_kv4_append(s["cache"], s["k_new"], s["v_new"], s["slots"], s["rows"])
        native.sd_kv4_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if case["op"] == "read":
        native.sd_kv4_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if case["op"] == "rope":
        if case["cache"]:
            native.sd_rope_append(s["rope"], s["pos"], s["q"], s["k"], s["v"], s["q_out"], None, s["k_cache"],
                                  s["v_cache"], s["slots"], interleaved=case["interleaved"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        native.sd_rope_append(s["rope"], s["pos"], s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"],
                              interleaved=case["interleaved"])
        return s["q_out"], s["k_out"]
    native.sd_logprobs(s["logits"], s["given"], s["lp"], s["ids"], s["top_lp"], s["entropy"], s["lse"],
                       temperature=case["temperature"], workspace=s["ws"])
    return s["lp"], s["ids"], s["top_lp"], s["entropy"], s["lse"]


# ------------------------------------------------------------------------------------------ plain forms

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
    block = lambda x: x.float()[at].transpose(1, 2)                   # noqa: E731
    pos = torch.arange(table.shape[1] * PAGE, device=DEVICE)
    q_pos = ctx[:, None] + depth                                       # [batch, nmax]
    k_pos = torch.cat([pos.expand(batch, -1), q_pos], 1)
    cached = pos < ctx[:, None]
    mask = torch.cat([cached[:, None, :].expand(-1, nmax, -1), (seen > 0) & is_node[:, None, :]], 2)
    if case["window"]:
        mask = mask & (k_pos[:, None, :] > q_pos[:, :, None] - case["window"])
    rows = q[at].reshape(batch, nmax, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, dim)
    k, v = (x.transpose(1, 2).reshape(batch, hkv, -1, dim) for x in _values(s["cache"][table], dim))
    score = rows @ torch.cat([k, block(s["k_new"])], 2).transpose(2, 3)
    score = score.reshape(batch, hkv, hq // hkv, nmax, -1) / math.sqrt(dim)
    del k
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    if s["slopes"] is not None:
        away = (k_pos[:, None, :] - q_pos[:, :, None]).float()
        score = score + s["slopes"].reshape(hkv, hq // hkv, 1, 1) * away[:, None, None]
    score = torch.where(mask[:, None, None], score, float("-inf"))
    w = torch.exp(score - score.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    v = torch.cat([v.masked_fill(~cached[:, None, :, None], 0.0), block(s["v_new"])], 2)
    out = w.reshape(batch, hkv, -1, w.shape[-1]) @ v
    out = out.reshape(batch, hkv, hq // hkv, nmax, dim).permute(0, 3, 1, 2, 4).reshape(batch, nmax, hq, dim)
    return out[is_node].bfloat16()


def _plain_append(s, case):
    """Codes and scales of the rows, set into their pages; then what the cache holds for them."""
    live = s["slots"] >= 0
    slots = s["slots"].long()[live]
    src = s["rows"].long()[live] if s["rows"] is not None else torch.arange(s["slots"].numel(), device=DEVICE)[live]
    page, t, dim, cut = slots // PAGE, slots % PAGE, case["dim"], 8 * case["dim"]
    k, v, nb = s["cache"][..., 0, :], s["cache"][..., 1, :], case["dim"] // BLOCK
    ck, sk = _codes_and_scales(s["k_new"][:, src].float())                    # [layers, rows, heads, dim]
    cv, sv = _codes_and_scales(s["v_new"][:, src].float())
    # K: a token's 16 bytes of every block, its scales
    at = (torch.arange(nb, device=DEVICE)[:, None] * 256 + torch.arange(16, device=DEVICE)).reshape(-1) + t[:, None] * 16
    at = torch.cat([at, cut + t[:, None] * 2 * nb + torch.arange(2 * nb, device=DEVICE)], 1)
    layers, heads = torch.arange(case["layers"], device=DEVICE)[:, None, None, None], torch.arange(case["hkv"], device=DEVICE)
    where = (layers, page[:, None, None], heads[:, None])
    k[(*where, at[:, None])] = torch.cat([_words(ck), sk.view(torch.uint8)], -1)
    # V: a nibble of every dim's 8 bytes, two bytes of every block's scales; the nibbles of a byte one after the other
    d = torch.arange(dim, device=DEVICE) * 8
    byte, shift = (t // 8) * 4 + (t % 2) * 2 + (t % 8) // 4, (t % 4 // 2) * 4
    for low in (0, 4):
        mine = shift == low
        put = (layers, page[mine][:, None, None], heads[:, None], (d + byte[mine][:, None])[:, None])
        v[put] = (v[put] & (240 if low == 0 else 15)) | (cv[:, mine] << low).to(torch.uint8)
    at = cut + torch.arange(nb, device=DEVICE)[:, None] * 32 + torch.arange(2, device=DEVICE)
    v[(*where, (at.reshape(-1) + 2 * t[:, None])[:, None])] = sv.view(torch.uint8)
    return _plain_read(s, case)


def _plain_read(s, case):
    live = s["slots"] >= 0
    slots = s["slots"].long()[live]
    k, v = _values(s["cache"][:, slots // PAGE], case["dim"])                 # [layers, rows, heads, 16, dim]
    t = (slots % PAGE)[None, :, None, None, None].expand(case["layers"], -1, case["hkv"], 1, case["dim"])
    s["k_out"][:, live], s["v_out"][:, live] = (x.gather(3, t)[:, :, :, 0].bfloat16() for x in (k, v))
    return s["k_out"], s["v_out"]


def _rotated(x, table, interleaved):
    x, half = x.float(), table.shape[1] // 2
    c, sn = table[:, None, :half], table[:, None, half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, x[..., 2 * half:]], -1).bfloat16()


def _plain_rope(s, case):
    table = s["rope"][s["pos"].long()]
    q, k = (_rotated(s[c], table, case["interleaved"]) for c in "qk")
    if not case["cache"]:
        return q, k
    slots = s["slots"].long()
    s["k_cache"][slots // PAGE, :, slots % PAGE], s["v_cache"][slots // PAGE, :, slots % PAGE] = k, s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_logprobs(s, case):
    z = s["logits"].float() / case["temperature"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    entropy = (torch.log(total) - (e * (z - m)).sum(1, keepdim=True) / total)[:, 0]
    given = None if s["given"] is None else z.gather(1, s["given"].long()) - lse
    if not case["top"]:
        return given, None, None, entropy, lse[:, 0]
    del e
    # largest first, ties by the lower index: one whole number for both (the bits of a float order as it does)
    bits = (s["logits"].float() + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, (bits & 0x7fffffff).neg()) * (1 << 20)
    key = key - torch.arange(case["vocab"], device=DEVICE)
    ids = key.topk(case["top"], 1)[1]
    return given, ids.int(), z.gather(1, ids) - lse, entropy, lse[:, 0]


# ------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "read": _exact_read, "rope": _exact_rope,
            "logprobs": _exact_logprobs}[case["op"]](s, case)


def _held(cache, pages, g, dim):
    """K and V of KV head g in these pages, float64 [len(pages) * 16, dim], byte by byte."""
    def signed(b):           # two codes of a byte, low one first
        return torch.stack([b & 15, b >> 4], -1).double() - 8

    def scales(raw):
        w = raw.reshape(-1, 2).int()
        return (w[:, 0] | w[:, 1] << 8).to(torch.int16).view(torch.bfloat16).double()
    rec, n, nb = cache[pages, g], len(pages), dim // BLOCK
    k, v = rec[:, 0], rec[:, 1]
    # bytes of a word: codes (0, 2), (4, 6), (1, 3), (5, 7)
    order = [0, 4, 1, 5, 2, 6, 3, 7]
    ck = signed(k[:, :8 * dim].reshape(n, nb, PAGE, 4, 4)).reshape(n, nb, PAGE, 4, 8)[..., order]
    ck = ck.permute(0, 2, 1, 3, 4).reshape(n, PAGE, nb, BLOCK)
    cv = signed(v[:, :8 * dim].reshape(n, dim, 2, 4)).reshape(n, dim, 2, 8)[..., order].reshape(n, nb, BLOCK, PAGE)
    ck = ck * scales(k[:, 8 * dim:]).reshape(n, PAGE, nb, 1)
    cv = cv * scales(v[:, 8 * dim:]).reshape(n, nb, 1, PAGE)
    return ck.reshape(-1, dim), cv.reshape(n, dim, PAGE).transpose(1, 2).reshape(-1, dim)


def _exact_attn(s, case):
    """One sequence, one KV head at a time; the scores of each node over its own keys."""
    group, parents, dim = case["hq"] // case["hkv"], s["parents"].tolist(), case["dim"]
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
            k, v = _held(s["cache"], pages, g, dim)
            k = torch.cat([k[:n], s["k_new"][lo:hi, g].double()])
            v = torch.cat([v[:n], s["v_new"][lo:hi, g].double()])
            q = s["q"][lo:hi, g * group:(g + 1) * group].double()
            t = torch.einsum("nhd,kd->hnk", q, k) * dim ** -0.5
            if case["softcap"]:
                t = torch.tanh(t / case["softcap"]) * case["softcap"]
            if s["slopes"] is not None:
                t += s["slopes"][g * group:(g + 1) * group].double()[:, None, None] * away
            t = torch.softmax(t.masked_fill(~see, -math.inf), -1)
            out[lo:hi, g * group:(g + 1) * group] = torch.einsum("hnk,kd->nhd", t, v)
    return out


def _exact_append(s, case):
    """The rows as the cache holds them: each block on its own grid, from the definition."""
    slots = s["slots"].tolist()
    out = []
    for c in "kv":
        got = torch.zeros(s[c + "_out"].shape, dtype=torch.float64, device=DEVICE)
        src = s["rows"] if s["rows"] is not None else torch.arange(len(slots), device=DEVICE)
        n = sum(x >= 0 for x in slots)                       # the rows lie in front
        x = s[c + "_new"][:, src[:n].long()].double()
        x = x.reshape(*x.shape[:-1], -1, BLOCK)
        big = x.abs().amax(-1, keepdim=True)
        first = torch.where(x.abs() == big, torch.arange(BLOCK, device=DEVICE), BLOCK).amin(-1, keepdim=True)
        s8 = -x.gather(-1, first) / 8
        unit = torch.exp2(torch.floor(torch.log2(s8.abs().clamp(min=2.0 ** -120))) - 4)
        s8 = torch.round(s8 / unit) * unit
        s8 = torch.where(big < 2.0 ** -100, 0.0, s8)
        code = torch.round(x / torch.where(s8 == 0, 1.0, s8)).clamp(-8, 7)
        got[:, :n] = (code * s8).flatten(-2)
        out.append(got)
    return out


def _exact_read(s, case):
    k, v = (torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEVICE) for _ in "kv")
    slots = s["slots"][s["slots"] >= 0].long()
    for layer in range(case["layers"]):
        for g in range(case["hkv"]):
            hk, hv = _held(s["cache"][layer], torch.unique(slots // PAGE), g, case["dim"])
            at = torch.searchsorted(torch.unique(slots // PAGE), slots // PAGE) * PAGE + slots % PAGE
            k[layer, :len(slots), g], v[layer, :len(slots), g] = hk[at], hv[at]
    return k, v


def _exact_rope(s, case):
    def turned(x):
        x, half = x.double(), case["rot"] // 2
        pair = [2 * i for i in range(half)] if case["interleaved"] else list(range(half))
        mate = [p + 1 for p in pair] if case["interleaved"] else [p + half for p in pair]
        y, t = x.clone(), s["rope"].double()[s["pos"].long()]
        z = torch.complex(x[..., pair], x[..., mate]) * torch.complex(t[:, None, :half], t[:, None, half:])
        y[..., pair], y[..., mate] = z.real, z.imag
        return y
    q, k = turned(s["q"]), turned(s["k"])
    if not case["cache"]:
        return q, k
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for rows, cache in ((k, kc), (s["v"].double(), vc)):
        flat = cache.transpose(1, 2).flatten(0, 1).contiguous()               # a row for each slot
        flat[s["slots"].long()] = rows
        cache.copy_(flat.unflatten(0, (-1, PAGE)).transpose(1, 2))
    return q, kc, vc


def _exact_logprobs(s, case):
    given, top, entropy, norm = [], [], [], []
    for r in range(0, case["rows"], 128):
        z = s["logits"][r:r + 128].double() / case["temperature"]
        p = torch.log_softmax(z, 1)
        norm.append(torch.logsumexp(z, 1))
        entropy.append(-(p.exp() * p).sum(1))
        if s["given"] is not None:
            given.append(p.gather(1, s["given"][r:r + 128].long()))
        if case["top"]:
            top.append(torch.sort(p, 1, descending=True)[0][:, :case["top"]])
    cat = lambda x: torch.cat(x) if x else None  # noqa: E731
    return cat(given), None, cat(top), cat(entropy), cat(norm)


# ------------------------------------------------------------------------------------------ the work of a pass

def work(case):
    if case["op"] == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        size = rows * vocab * (4 if case["dtype"] == "float32" else 2)
        return {"bytes": size + rows * (8 + 8 * case["given"] + 8 * case["top"]), "flops": 5 * rows * vocab}
    if case["op"] == "attn":
        lens, nodes = _lens(case, case["ctx_lo"], case["ctx_hi"], 1), [len(t) for t in _trees(case)]
        spans = [min(n, case["window"] - 1) if case["window"] else n for n in lens]
        row = case["hkv"] * case["dim"]
        total, pages = sum(nodes), sum(-(-n // PAGE) for n in spans)
        size = sum(spans) * row * 9 // 8 + 4 * pages + total * (4 * case["hq"] * case["dim"] + 4 * row)
        flops = sum(4 * n * case["hq"] * case["dim"] * (span + 1) for n, span in zip(nodes, spans))
        return {"bytes": size, "flops": flops}
    add = sum(_lens(case, case["rows_lo"], case["rows_hi"], 3))
    row = case["hkv"] * case["dim"]
    if case["op"] == "rope":
        q = case["hq"] * case["dim"]
        moved = add * (4 * q + 4 * row + (4 * row if case["cache"] else 0) + 4 * case["rot"] + 8)
        return {"bytes": moved, "flops": 3 * add * (case["hq"] + case["hkv"]) * case["rot"]}
    packed, plain = case["layers"] * add * row * 9 // 8, case["layers"] * add * row * 4
    size = 2 * packed + 2 * plain if case["op"] == "append" else packed + plain
    return {"bytes": size + 4 * (add + 5), "flops": 4 * case["layers"] * add * row}
