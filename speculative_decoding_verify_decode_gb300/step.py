"""One verify step on the GPU: every layer's attention, then accept, then commit.

The three C-ABI calls run in order on one CUDA stream with no host
synchronisation between them, so a step can also be captured into a CUDA
graph (``VerifyStep.capture``).  This module owns the output buffers and the
workspaces; the inputs (queries, draft K/V, caches, logits, tree, page
table) belong to the caller.  ``Kv8Cache`` and ``Kv8Step`` are the same over
the 8-bit block-scaled cache, with its pages allocated on the GPU, ``Kv4Cache`` and ``Kv4Step`` over the 4-bit one.
"""
from __future__ import annotations

import numpy as np
import torch

from . import native


class VerifyStep:
    """Buffers and calls for one verify step of a fixed batch shape."""

    def __init__(self, q_indptr, max_pages_per_seq: int, num_pool_pages: int, num_layers: int, vocab: int,
                 device="cuda", num_splits: int = 0, max_path: int | None = None, want_lse: bool = False,
                 window: int = 0, k_scales=None, v_scales=None):
        """``k_scales`` / ``v_scales`` (per-layer floats) select e4m3 caches: attention reads the codes with
        these scales and the commit quantises the accepted rows with them."""
        self.q_indptr = np.asarray(q_indptr, dtype=np.int32)
        self.batch = len(self.q_indptr) - 1
        self.total = int(self.q_indptr[-1])
        self.num_layers = int(num_layers)
        self.vocab = int(vocab)
        self.device = torch.device(device)
        self.shape = native.Shape(self.q_indptr, max_pages_per_seq, num_pool_pages, num_splits, window)
        # layers after the first follow the previous layer's attention, which writes no context state
        self.shape_next = self.shape.with_ctx_stable(True)
        self.fp8 = k_scales is not None
        if self.fp8 and (v_scales is None or len(k_scales) != self.num_layers or len(v_scales) != self.num_layers):
            raise ValueError("e4m3 caches need one K and one V scale per layer")
        self.k_scales = None if k_scales is None else [float(x) for x in k_scales]
        self.v_scales = None if v_scales is None else [float(x) for x in v_scales]
        self.max_path = int(max_path or int(np.diff(self.q_indptr).max()))
        dev = self.device
        ws = native.sd_verify_attn_workspace_size(self.shape)
        self.attn_ws = torch.empty(max(ws, 1), dtype=torch.uint8, device=dev)
        self.acc_ws = torch.empty(max(native.sd_accept_workspace_size(self.q_indptr, self.vocab), 1),
                                  dtype=torch.uint8, device=dev)
        self.out = [torch.empty((self.total, 24, 256), dtype=torch.bfloat16, device=dev)
                    for _ in range(self.num_layers)]
        self.lse = ([torch.empty((self.total, 24), dtype=torch.float32, device=dev)
                     for _ in range(self.num_layers)] if want_lse else None)
        self.accept_len = torch.empty(self.batch, dtype=torch.int32, device=dev)
        self.path = torch.empty((self.batch, self.max_path), dtype=torch.int32, device=dev)
        self.out_tokens = torch.empty((self.batch, self.max_path), dtype=torch.int32, device=dev)
        self.target_tokens = torch.empty(self.total, dtype=torch.int32, device=dev)
        self.new_ctx_lens = torch.empty(self.batch, dtype=torch.int32, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)

    def attention(self, layer, q, k_cache, v_cache, k_new, v_new, page_table, ctx_lens, parents, stream=None,
                  ctx_stable: bool = False):
        """One layer's attention.  ``ctx_stable``: the previous kernel on the stream writes no context state
        (sd_shape.ctx_stable), so the context loads may start before it finishes."""
        lse = None if self.lse is None else self.lse[layer]
        shape = self.shape_next if ctx_stable else self.shape
        if self.fp8:
            native.sd_verify_attn_fp8(shape, q, k_cache, v_cache, self.k_scales[layer], self.v_scales[layer],
                                      k_new, v_new, page_table, ctx_lens, parents, self.out[layer], lse,
                                      self.attn_ws, self.dev_status, stream)
        else:
            native.sd_verify_attn(shape, q, k_cache, v_cache, k_new, v_new, page_table, ctx_lens, parents,
                                  self.out[layer], lse, self.attn_ws, self.dev_status, stream)

    def accept(self, logits, parents, draft_tokens, stream=None):
        native.sd_accept(self.q_indptr, self.vocab, logits, parents, draft_tokens, self.accept_len, self.path,
                         self.out_tokens, self.target_tokens, self.max_path, self.acc_ws, self.dev_status,
                         stream)

    def commit(self, k_caches, v_caches, k_news, v_news, page_table, ctx_lens, stream=None):
        if self.fp8:
            native.sd_kv_commit_fp8(self.shape, k_caches, v_caches, self.k_scales, self.v_scales, k_news, v_news,
                                    page_table, ctx_lens, self.new_ctx_lens, self.accept_len, self.path,
                                    self.max_path, self.dev_status, stream)
            return
        native.sd_kv_commit(self.shape, k_caches, v_caches, k_news, v_news, page_table, ctx_lens,
                            self.new_ctx_lens, self.accept_len, self.path, self.max_path, self.dev_status,
                            stream)

    def run(self, q, k_caches, v_caches, k_news, v_news, page_table, ctx_lens, parents, draft_tokens, logits,
            stream=None, commit: bool = True):
        """q/k_caches/v_caches/k_news/v_news are per-layer lists of device tensors."""
        for layer in range(self.num_layers):
            self.attention(layer, q[layer], k_caches[layer], v_caches[layer], k_news[layer], v_news[layer],
                           page_table, ctx_lens, parents, stream, ctx_stable=layer > 0)
        self.accept(logits, parents, draft_tokens, stream)
        if commit:
            self.commit(k_caches, v_caches, k_news, v_news, page_table, ctx_lens, stream)

    def launches_per_step(self, commit: bool = True) -> int:
        """Kernel launches one ``run`` issues (attention split (+ merge), argmax, accept, commit)."""
        merge = 1 if native.sd_verify_attn_workspace_size(self.shape) > 0 else 0
        return self.num_layers * (1 + merge) + 2 + (1 if commit else 0)

    def capture(self, *args, **kwargs) -> torch.cuda.CUDAGraph:
        """Capture ``run(*args, **kwargs)`` into a CUDA graph (inputs must stay at the same addresses)."""
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream(device=self.device)
        s.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                self.run(*args, stream=s, **kwargs)
        torch.cuda.current_stream(self.device).wait_stream(s)
        return g


def rope_table(length: int, rot_dim: int, theta: float = 1e6, device="cuda") -> torch.Tensor:
    """Cosines, then sines, of ``length`` positions for sd_rope_append, fp32 [length, rot_dim]; the angles are formed in
    64 bits (in 32 those of far positions lose their digits)."""
    dev = torch.device(device)
    freq = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=dev) / rot_dim)
    angle = torch.arange(length, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


class _PagedCache:
    """Page tables and the free list of a pool of pages, all on the GPU.

    ``extend`` takes pages for joining tokens and appends their K/V, ``release`` gives pages back; both only
    launch kernels, so a step that contains them can be captured into a CUDA graph and replayed.  The calls of one
    cache follow each other: they share its state and scratch, so on two streams an event has to order them.
    """

    def _init_pages(self, batch: int, max_pages_per_seq: int, num_pool_pages: int):
        dev, self.num_pool_pages = self.device, int(num_pool_pages)
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
        self.page_table = torch.full((batch, max_pages_per_seq), -1, dtype=torch.int32, device=dev)
        self.ctx_lens, self.held, self.free_count = ints(batch), ints(batch), ints(1)
        self.free_list = torch.arange(num_pool_pages - 1, -1, -1, dtype=torch.int32, device=dev)
        self.free_count.fill_(num_pool_pages)
        self._new = ints(batch), ints(batch), ints(1)
        self.dev_status, self._said = ints(1), ints(1)

    def _on(self, stream):
        """The context of a stream: a torch stream, a raw handle, or None for the current one."""
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, self.device) if stream else torch.cuda.default_stream(self.device)
        return torch.cuda.stream(stream)

    def _settle(self, ctx: bool):
        new_ctx, new_held, new_count = self._new
        if ctx:
            self.ctx_lens.copy_(new_ctx)
        self.held.copy_(new_held)
        self.free_count.copy_(new_count)

    def extend(self, add_lens, k_new, v_new, slots, rows=None, q_indptr=None, path=None, stream=None):
        """``add_lens`` tokens join every sequence: their pages, then their rows of every layer's ``k_new`` and
        ``v_new`` into the cache.  ``slots`` (and ``rows`` with a path) are int32 scratch with room for all rows."""
        with self._on(stream):
            new_ctx, new_held, new_count = self._new
            native.sd_pages_extend(self.ctx_lens, add_lens, self.page_table, self.held, new_held, self.free_list,
                                   self.free_count, new_count, slots, rows=rows, new_ctx_lens=new_ctx,
                                   q_indptr=q_indptr, path=path, dev_status=self.dev_status)
            self._append(k_new, v_new, slots, rows)
            self._settle(ctx=True)

    def release(self, keep_lens, stream=None):
        """Every sequence keeps its first ``keep_lens`` tokens at most; the pages behind them become free.  A call that
        is refused (see sd_pages_release) leaves everything as it was."""
        with self._on(stream):
            _, new_held, new_count = self._new
            said = self._said.zero_()
            native.sd_pages_release(keep_lens, self.page_table, self.held, new_held, self.free_list, self.free_count,
                                    new_count, said)
            # refused: a status, and no page moved (a page whose id is out of range is reported, and moves)
            refused = (said != 0) & (new_count == self.free_count)
            self._settle(ctx=False)
            torch.minimum(self.ctx_lens, torch.where(refused, self.ctx_lens, keep_lens), out=self.ctx_lens)
            self.dev_status |= said


class Kv8Cache(_PagedCache):
    """A pool of 8-bit block-scaled K/V pages for every layer, its page tables, and the free list, all on the GPU."""

    def __init__(self, batch: int, max_pages_per_seq: int, num_pool_pages: int, num_layers: int,
                 num_kv_heads: int = 4, head_dim: int = 256, device="cuda"):
        dev = torch.device(device)
        codes = (num_layers, num_pool_pages, num_kv_heads, 16, head_dim)
        self.k, self.v = (torch.zeros(codes, dtype=torch.uint8, device=dev) for _ in "kv")
        self.device = self.k.device       # "cuda" is the device that is current now
        self.k_scales, self.v_scales = (torch.ones(codes[:3], dtype=torch.float32, device=self.device) for _ in "kv")
        self._init_pages(batch, max_pages_per_seq, num_pool_pages)

    def _append(self, k_new, v_new, slots, rows):
        native.sd_kv8_append(self.k, self.v, self.k_scales, self.v_scales, k_new, v_new, slots, rows, self.dev_status)


class Kv4Cache(_PagedCache):
    """The same with 4-bit pages: ``kv`` uint8 [layers, pool, heads, 2, 9 * dim] (include/sd_kv4.h)."""

    def __init__(self, batch: int, max_pages_per_seq: int, num_pool_pages: int, num_layers: int,
                 num_kv_heads: int = 4, head_dim: int = 256, device="cuda"):
        shape = native.kv4_cache_shape(num_pool_pages, num_kv_heads, head_dim)
        self.kv = torch.zeros((num_layers, *shape), dtype=torch.uint8, device=torch.device(device))
        self.device = self.kv.device      # "cuda" is the device that is current now
        self._init_pages(batch, max_pages_per_seq, num_pool_pages)

    def _append(self, k_new, v_new, slots, rows):
        native.sd_kv4_append(self.kv, k_new, v_new, slots, rows, self.dev_status)

    def read(self, slots, k_out, v_out, stream=None):
        """The values at these slots, every layer's, as bf16 rows (sd_kv4_read)."""
        native.sd_kv4_read(self.kv, slots, k_out, v_out, self.dev_status, stream)


class Kv8Step:
    """One verify step over a Kv8Cache: every layer's attention, accept, the accepted path's pages and append."""

    def __init__(self, cache: Kv8Cache, q_indptr, vocab: int, num_q_heads: int = 24, window: int = 0,
                 softcap: float = 0.0, slopes=None, max_path: int | None = None):
        self.cache, self.vocab, self.softcap, self.slopes = cache, int(vocab), softcap, slopes
        self.q_indptr = np.asarray(q_indptr, dtype=np.int32)
        layers, pool, heads, dim = self._geometry()
        batch, total, dev = len(self.q_indptr) - 1, int(self.q_indptr[-1]), cache.device
        self.shape = native.Shape(self.q_indptr, cache.page_table.shape[1], pool, window=window,
                                  num_q_heads=num_q_heads, num_kv_heads=heads, head_dim=dim)
        self.max_path = int(max_path or int(np.diff(self.q_indptr).max()))
        byte = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
        self.attn_ws = byte(self._workspace_size())
        self.acc_ws = byte(native.sd_accept_workspace_size(self.q_indptr, self.vocab))
        ints = lambda *s: torch.empty(s, dtype=torch.int32, device=dev)
        self.out = torch.empty((layers, total, num_q_heads, dim), dtype=torch.bfloat16, device=dev)
        self.accept_len, self.target_tokens = ints(batch), ints(total)
        self.path, self.out_tokens = ints(batch, self.max_path), ints(batch, self.max_path)
        self.slots, self.rows = ints(total), ints(total)

    def _geometry(self):
        layers, pool, heads, _, dim = self.cache.k.shape
        return layers, pool, heads, dim

    def _workspace_size(self):
        return native.sd_kv8_attn_workspace_size(self.shape)

    def attention(self, layer, q, k_new, v_new, parents, stream=None):
        c = self.cache
        native.sd_kv8_attn(self.shape, q, c.k[layer], c.v[layer], c.k_scales[layer], c.v_scales[layer], k_new, v_new,
                           c.page_table, c.ctx_lens, parents, self.out[layer], softcap=self.softcap,
                           slopes=self.slopes, workspace=self.attn_ws, dev_status=c.dev_status, stream=stream)

    def run(self, q, k_new, v_new, parents, draft_tokens, logits, stream=None):
        """q, k_new and v_new are per-layer lists (or tensors with a leading layer dimension)."""
        # sd_accept takes the current device's stream; the other calls go by their tensors
        with torch.cuda.device(self.cache.device):
            for layer in range(len(q)):
                self.attention(layer, q[layer], k_new[layer], v_new[layer], parents, stream)
            native.sd_accept(self.q_indptr, self.vocab, logits, parents, draft_tokens, self.accept_len, self.path,
                             self.out_tokens, self.target_tokens, self.max_path, self.acc_ws, self.cache.dev_status,
                             stream)
            self.cache.extend(self.accept_len, k_new, v_new, self.slots, self.rows, self.q_indptr, self.path, stream)


class Kv4Step(Kv8Step):
    """One verify step over a Kv4Cache; with ``top`` it also leaves every node's log probabilities: of the target's own
    choice (``logprobs`` [nodes, 1]; the emitted tokens' are the rows of the accepted path) and of its ``top`` likeliest
    tokens (``top_ids``, ``top_logprobs``), and the entropy."""

    def __init__(self, cache: Kv4Cache, q_indptr, vocab: int, num_q_heads: int = 24, window: int = 0, softcap: float = 0.0,
                 slopes=None, max_path: int | None = None, top: int = 0):
        if not 0 <= top <= min(int(vocab), native.SD_LOGPROBS_MAX_TOP):
            raise ValueError(f"top is 0..{min(int(vocab), native.SD_LOGPROBS_MAX_TOP)}")
        super().__init__(cache, q_indptr, vocab, num_q_heads, window, softcap, slopes, max_path)
        self.top, total, dev = int(top), int(self.q_indptr[-1]), cache.device
        layers, _, heads, dim = self._geometry()
        self.q_turned, self.k_turned = (torch.empty((layers, total, h, dim), dtype=torch.bfloat16, device=dev)
                                        for h in (num_q_heads, heads))
        if self.top:
            f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)
            self.logprobs, self.top_logprobs, self.entropy = f32(total, 1), f32(total, self.top), f32(total)
            self.top_ids = torch.empty((total, self.top), dtype=torch.int32, device=dev)
            self.lp_ws = torch.empty(max(16, native.sd_logprobs_workspace_size(total, self.vocab, self.top)),
                                     dtype=torch.uint8, device=dev)

    def _geometry(self):
        layers, pool, heads, _, width = self.cache.kv.shape
        return layers, pool, heads, width // 9

    def _workspace_size(self):
        return native.sd_kv4_attn_workspace_size(self.shape)

    def attention(self, layer, q, k_new, v_new, parents, stream=None):
        c = self.cache
        native.sd_kv4_attn(self.shape, q, c.kv[layer], k_new, v_new, c.page_table, c.ctx_lens, parents, self.out[layer],
                           softcap=self.softcap, slopes=self.slopes, workspace=self.attn_ws, dev_status=c.dev_status,
                           stream=stream)

    def run(self, q, k_new, v_new, parents, draft_tokens, logits, stream=None, rope=None):
        """As Kv8Step.run; ``rope`` = (table, positions of the nodes) turns q and k_new first."""
        status = self.cache.dev_status
        if rope is not None:
            table, positions = rope
            for layer in range(len(q)):
                native.sd_rope_append(table, positions, q[layer], k_new[layer], q_out=self.q_turned[layer],
                                      k_out=self.k_turned[layer], dev_status=status, stream=stream)
            q, k_new = self.q_turned, self.k_turned
        super().run(q, k_new, v_new, parents, draft_tokens, logits, stream)
        if self.top:
            native.sd_logprobs(logits, self.target_tokens[:, None], self.logprobs, self.top_ids, self.top_logprobs,
                               self.entropy, workspace=self.lp_ws, dev_status=status, stream=stream)


def device_inputs(w, device="cuda"):
    """Move a synthetic workload's small host arrays to the device (int32)."""
    dev = torch.device(device)
    as_t = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)
    return dict(page_table=as_t(w.page_table), ctx_lens=as_t(w.ctx_lens), parents=as_t(w.parents),
                draft_tokens=as_t(w.draft_tokens))
