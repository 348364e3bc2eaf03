"""ctypes binding of libsdverify.so (include/sd_verify.h, sd_gdn.h, sd_kv8.h, sd_kv4.h, sd_rope.h, sd_logprobs.h).

Argument marshalling only: every function here turns torch tensors into the
device pointers and host arrays of the C ABI and raises on a non-zero status.
All computation happens in the library's CUDA kernels.  There is no fallback:
if the library is missing or was not built for this GPU, the first call
raises.
"""
from __future__ import annotations

import ctypes
import os
from array import array

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsdverify.so")

SD_OK, SD_ERR_INVALID_ARG, SD_ERR_UNSUPPORTED, SD_ERR_CUDA, SD_ERR_WORKSPACE = range(5)
SD_DEV_BAD_PARENTS = 1
SD_DEV_BAD_PAGE = 2
SD_DEV_BAD_CTX = 4
SD_DEV_BAD_ACCEPT = 8
SD_DEV_NAN_LOGITS = 16
SD_DEV_PATH_OVERFLOW = 32
SD_DEV_TIMEOUT = 64
SD_DEV_NO_PAGES = 128
SD_DEV_BAD_SCALE = 256
SD_DEV_BAD_SLOT = 512
SD_DEV_NOT_FINITE = 1024
SD_DEV_BAD_POSITION = 2048
SD_LOGPROBS_MAX_TOP = 32
MAX_NODES = 64
MAX_BATCH = 256
MAX_LAYERS = 64


class SdShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("q_indptr_h", ctypes.POINTER(ctypes.c_int)),
                ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_pages_per_seq", ctypes.c_int), ("num_pool_pages", ctypes.c_int),
                ("num_splits", ctypes.c_int),
                ("window", ctypes.c_int), ("ctx_stable", ctypes.c_int)]


class SdGdnShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("q_indptr_h", ctypes.POINTER(ctypes.c_int)),
                ("num_k_heads", ctypes.c_int), ("num_v_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class SdKv8Opts(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong), ("v_stride", ctypes.c_longlong)]


class SdRopeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("num_rows", "num_q_heads", "num_kv_heads", "head_dim", "rot_dim", "interleaved",
                                            "table_len", "page_size", "num_pool_pages")] + \
               [(n, ctypes.c_longlong) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride", "k_out_stride")]


class SdError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def load() -> ctypes.CDLL:
    """Load (once) and type the library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m speculative_decoding_verify_decode_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, ip, fp, sz = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int), ctypes.c_void_p, ctypes.c_size_t
    shp = ctypes.POINTER(SdShape)
    lib.sd_status_string.restype = ctypes.c_char_p
    lib.sd_status_string.argtypes = [ctypes.c_int]
    lib.sd_verify_attn_workspace_size.restype = sz
    lib.sd_verify_attn_workspace_size.argtypes = [shp]
    lib.sd_verify_attn.restype = ctypes.c_int
    lib.sd_verify_attn.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, vp, vp, fp, vp, sz, vp, vp]
    lib.sd_verify_attn_fp8.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.sd_verify_attn_fp8.argtypes = [shp, vp, vp, vp, f32, f32, vp, vp, vp, vp, vp, vp, fp, vp, sz, vp, vp]
    lib.sd_verify_attn_noalloc.restype = ctypes.c_int
    lib.sd_verify_attn_noalloc.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, vp, vp, fp, vp, vp]
    lib.sd_accept_workspace_size.restype = sz
    lib.sd_accept_workspace_size.argtypes = [ctypes.c_int, ip, ctypes.c_int]
    lib.sd_accept.restype = ctypes.c_int
    lib.sd_accept.argtypes = [ctypes.c_int, ip, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                              vp, sz, vp, vp]
    lib.sd_sample_accept_workspace_size.restype = sz
    lib.sd_sample_accept_workspace_size.argtypes = [ctypes.c_int, ip, ctypes.c_int]
    lib.sd_sample_accept.restype = ctypes.c_int
    lib.sd_sample_accept.argtypes = [ctypes.c_int, ip, ctypes.c_int, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp,
                                     vp, ctypes.c_int, vp, sz, vp, vp]
    lib.sd_kv_commit.restype = ctypes.c_int
    pp = ctypes.POINTER(ctypes.c_void_p)
    lib.sd_kv_commit.argtypes = [shp, ctypes.c_int, pp, pp, pp, pp, vp, vp, vp, vp, vp, ctypes.c_int, vp, vp]
    lib.sd_kv_commit_fp8.restype = ctypes.c_int
    fpp = ctypes.POINTER(ctypes.c_float)
    lib.sd_kv_commit_fp8.argtypes = [shp, ctypes.c_int, pp, pp, fpp, fpp, pp, pp, vp, vp, vp, vp, vp, ctypes.c_int,
                                     vp, vp]
    gshp = ctypes.POINTER(SdGdnShape)
    lib.sd_gdn_tree_cache_size.restype = sz
    lib.sd_gdn_tree_cache_size.argtypes = [gshp]
    lib.sd_gdn_conv_tree.restype = ctypes.c_int
    lib.sd_gdn_conv_tree.argtypes = [ctypes.c_int, ip, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp]
    lib.sd_gdn_tree.restype = ctypes.c_int
    lib.sd_gdn_tree.argtypes = [gshp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.sd_gdn_commit.restype = ctypes.c_int
    lib.sd_gdn_commit.argtypes = [gshp, ctypes.c_int, pp, pp, ctypes.c_int, pp, pp, vp, vp, ctypes.c_int, vp, vp]
    lib.sd_ddtree_workspace_size.restype = sz
    lib.sd_ddtree_workspace_size.argtypes = [ctypes.c_int] * 4
    lib.sd_ddtree_build.restype = ctypes.c_int
    lib.sd_ddtree_build.argtypes = [ctypes.c_int] * 5 + [vp, vp, vp, vp, vp, vp, sz, vp, vp]
    i32, i64 = ctypes.c_int, ctypes.c_longlong
    lib.sd_pages_extend.restype = i32
    lib.sd_pages_extend.argtypes = [i32, i32, i32, vp, vp, ip, vp, i32, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp,
                                    vp, vp]
    lib.sd_pages_release.restype = i32
    lib.sd_pages_release.argtypes = [i32, i32, i32] + [vp] * 8 + [vp]
    lib.sd_kv8_append.restype = i32
    lib.sd_kv8_append.argtypes = [i32] * 5 + [vp] * 6 + [i64, i32, vp, vp, i32, vp, vp]
    lib.sd_kv8_attn_workspace_size.restype = sz
    lib.sd_kv8_attn_workspace_size.argtypes = [shp]
    lib.sd_kv8_attn.restype = i32
    lib.sd_kv8_attn.argtypes = [shp, ctypes.POINTER(SdKv8Opts)] + [vp] * 12 + [vp, sz, vp, vp]
    lib.sd_kv4_append.restype = i32
    lib.sd_kv4_append.argtypes = [i32] * 5 + [vp] * 3 + [i64, i32, vp, vp, i32, vp, vp]
    lib.sd_kv4_read.restype = i32
    lib.sd_kv4_read.argtypes = [i32] * 5 + [vp] * 3 + [i64, vp, i32, vp, vp]
    lib.sd_kv4_attn_workspace_size.restype = sz
    lib.sd_kv4_attn_workspace_size.argtypes = [shp]
    lib.sd_kv4_attn.restype = i32
    lib.sd_kv4_attn.argtypes = [shp, ctypes.POINTER(SdKv8Opts)] + [vp] * 9 + [vp, sz, vp, vp]
    lib.sd_rope_append.restype = i32
    lib.sd_rope_append.argtypes = [ctypes.POINTER(SdRopeShape)] + [vp] * 12
    lib.sd_logprobs_workspace_size.restype = sz
    lib.sd_logprobs_workspace_size.argtypes = [i32] * 3
    lib.sd_logprobs.restype = i32
    lib.sd_logprobs.argtypes = [i32, i32, i32, vp, i64, f32, i32, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().sd_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != SD_OK:
        raise SdError(status, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the verify library must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _indptr(q_indptr) -> ctypes.Array:
    arr = np.ascontiguousarray(np.asarray(q_indptr, dtype=np.int32))
    return (ctypes.c_int * len(arr))(*arr.tolist())


class Shape:
    """An sd_shape with its host q_indptr kept alive (head geometries other than 24/4/256: sd_kv8_attn and sd_kv4_attn)."""

    def __init__(self, q_indptr, max_pages_per_seq: int, num_pool_pages: int, num_splits: int = 0,
                 window: int = 0, ctx_stable: bool = False, num_q_heads: int = 24, num_kv_heads: int = 4,
                 head_dim: int = 256):
        self.indptr = _indptr(q_indptr)
        self.c = SdShape(len(self.indptr) - 1, ctypes.cast(self.indptr, ctypes.POINTER(ctypes.c_int)),
                         int(num_q_heads), int(num_kv_heads), int(head_dim), 16, int(max_pages_per_seq),
                         int(num_pool_pages), int(num_splits), int(window), int(bool(ctx_stable)))
        n, c = int(self.indptr[-1]) if len(self.indptr) else 0, self.c
        # shapes of the quantised caches' attention: q and out, k_new and v_new, codes, scales, page table, per sequence, per node
        self.dims = ((n, c.num_q_heads, c.head_dim), (n, c.num_kv_heads, c.head_dim),
                     (c.num_pool_pages, c.num_kv_heads, 16, c.head_dim), (c.num_pool_pages, c.num_kv_heads),
                     (c.batch, c.max_pages_per_seq), (c.batch,), (n,))

    def with_ctx_stable(self, ctx_stable: bool = True) -> "Shape":
        """The same shape with the context-stable launch flag set (see sd_shape.ctx_stable)."""
        c = self.c
        return Shape(list(self.indptr), c.max_pages_per_seq, c.num_pool_pages, c.num_splits, c.window,
                     ctx_stable, c.num_q_heads, c.num_kv_heads, c.head_dim)

    @property
    def ref(self):
        return ctypes.byref(self.c)


def sd_verify_attn_workspace_size(shape: Shape) -> int:
    return int(load().sd_verify_attn_workspace_size(shape.ref))


def sd_verify_attn(shape: Shape, q, k_cache, v_cache, k_new, v_new, page_table, ctx_lens, parents, out,
                   lse=None, workspace=None, dev_status=None, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().sd_verify_attn(shape.ref, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
                                 _ptr(page_table), _ptr(ctx_lens), _ptr(parents), _ptr(out), _ptr(lse),
                                 _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream)),
           "sd_verify_attn")


def sd_verify_attn_fp8(shape: Shape, q, k_cache, v_cache, k_scale: float, v_scale: float, k_new, v_new,
                       page_table, ctx_lens, parents, out, lse=None, workspace=None, dev_status=None,
                       stream=None) -> None:
    """sd_verify_attn over e4m3 caches (uint8 [pool, 4, 16, 256]) with per-tensor scales."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().sd_verify_attn_fp8(shape.ref, _ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale),
                                     float(v_scale), _ptr(k_new), _ptr(v_new), _ptr(page_table), _ptr(ctx_lens),
                                     _ptr(parents), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                     _ptr(dev_status), _stream(stream)),
           "sd_verify_attn_fp8")


NOALLOC_SCRATCH_BYTES = 16 << 20


def sd_verify_attn_noalloc(shape: Shape, q, k_cache, v_cache, k_new, v_new, page_table, ctx_lens, parents, out,
                           lse=None, dev_status=None, stream=None) -> None:
    """sd_verify_attn with the library's fixed scratch array instead of a caller workspace."""
    _check(load().sd_verify_attn_noalloc(shape.ref, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_new),
                                         _ptr(v_new), _ptr(page_table), _ptr(ctx_lens), _ptr(parents), _ptr(out),
                                         _ptr(lse), _ptr(dev_status), _stream(stream)),
           "sd_verify_attn_noalloc")


def sd_accept_workspace_size(q_indptr, vocab: int) -> int:
    ind = _indptr(q_indptr)
    return int(load().sd_accept_workspace_size(len(ind) - 1, ind, int(vocab)))


def sd_accept(q_indptr, vocab: int, logits, parents, draft_tokens, accept_len, path, out_tokens,
              target_tokens=None, max_path: int | None = None, workspace=None, dev_status=None,
              stream=None) -> None:
    ind = _indptr(q_indptr)
    if max_path is None:
        max_path = path.shape[-1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().sd_accept(len(ind) - 1, ind, int(vocab), _ptr(logits), _ptr(parents), _ptr(draft_tokens),
                            _ptr(accept_len), _ptr(path), _ptr(out_tokens), _ptr(target_tokens),
                            int(max_path), _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream)),
           "sd_accept")


def sd_sample_accept_workspace_size(q_indptr, vocab: int) -> int:
    ind = _indptr(q_indptr)
    return int(load().sd_sample_accept_workspace_size(len(ind) - 1, ind, int(vocab)))


def sd_sample_accept(q_indptr, vocab: int, temperature: float, logits, draft_probs, parents, draft_tokens, r_accept,
                     r_sample, accept_len, path, out_tokens, max_path: int | None = None, workspace=None,
                     dev_status=None, stream=None) -> None:
    """Sampling-based verification at temperature T (speculative sampling, multi-candidate on trees)."""
    ind = _indptr(q_indptr)
    if max_path is None:
        max_path = path.shape[-1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().sd_sample_accept(len(ind) - 1, ind, int(vocab), float(temperature), _ptr(logits), _ptr(draft_probs),
                                   _ptr(parents), _ptr(draft_tokens), _ptr(r_accept), _ptr(r_sample),
                                   _ptr(accept_len), _ptr(path), _ptr(out_tokens), int(max_path), _ptr(workspace),
                                   ws_bytes, _ptr(dev_status), _stream(stream)),
           "sd_sample_accept")


def _ptr_array(ts) -> ctypes.Array:
    return (ctypes.c_void_p * len(ts))(*[_ptr(t) for t in ts])


def sd_kv_commit(shape: Shape, k_cache_layers, v_cache_layers, k_new_layers, v_new_layers, page_table,
                 ctx_lens, new_ctx_lens, accept_len, path, max_path: int | None = None, dev_status=None,
                 stream=None) -> None:
    n = len(k_cache_layers)
    if not (len(v_cache_layers) == len(k_new_layers) == len(v_new_layers) == n):
        raise ValueError("per-layer pointer lists differ in length")
    if max_path is None:
        max_path = path.shape[-1]
    _check(load().sd_kv_commit(shape.ref, n, _ptr_array(k_cache_layers), _ptr_array(v_cache_layers),
                               _ptr_array(k_new_layers), _ptr_array(v_new_layers), _ptr(page_table),
                               _ptr(ctx_lens), _ptr(new_ctx_lens), _ptr(accept_len), _ptr(path),
                               int(max_path), _ptr(dev_status), _stream(stream)),
           "sd_kv_commit")


def sd_kv_commit_fp8(shape: Shape, k_cache_layers, v_cache_layers, k_scales, v_scales, k_new_layers,
                     v_new_layers, page_table, ctx_lens, new_ctx_lens, accept_len, path,
                     max_path: int | None = None, dev_status=None, stream=None) -> None:
    """sd_kv_commit into e4m3 caches: the accepted rows are quantised with the per-layer scales."""
    n = len(k_cache_layers)
    if not (len(v_cache_layers) == len(k_new_layers) == len(v_new_layers) == len(k_scales) == len(v_scales) == n):
        raise ValueError("per-layer lists differ in length")
    if max_path is None:
        max_path = path.shape[-1]
    ks = (ctypes.c_float * n)(*[float(x) for x in k_scales])
    vs = (ctypes.c_float * n)(*[float(x) for x in v_scales])
    _check(load().sd_kv_commit_fp8(shape.ref, n, _ptr_array(k_cache_layers), _ptr_array(v_cache_layers), ks, vs,
                                   _ptr_array(k_new_layers), _ptr_array(v_new_layers), _ptr(page_table),
                                   _ptr(ctx_lens), _ptr(new_ctx_lens), _ptr(accept_len), _ptr(path),
                                   int(max_path), _ptr(dev_status), _stream(stream)),
           "sd_kv_commit_fp8")


def sd_ddtree_workspace_size(batch: int, positions: int, vocab: int, topk: int) -> int:
    return int(load().sd_ddtree_workspace_size(int(batch), int(positions), int(vocab), int(topk)))


def sd_ddtree_build(draft_logits, topk: int, budget: int, root_tokens, parents, tokens, scores=None,
                    workspace=None, dev_status=None, stream=None) -> None:
    """draft_logits fp32 [batch, positions, vocab]; parents/tokens int32 [batch, 1 + budget]."""
    batch, positions, vocab = (int(x) for x in draft_logits.shape)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().sd_ddtree_build(batch, positions, vocab, int(topk), int(budget), _ptr(draft_logits),
                                  _ptr(root_tokens), _ptr(parents), _ptr(tokens), _ptr(scores), _ptr(workspace),
                                  ws_bytes, _ptr(dev_status), _stream(stream)),
           "sd_ddtree_build")


class GdnShape:
    """An sd_gdn_shape with its host q_indptr kept alive (head_dim 128)."""

    def __init__(self, q_indptr, num_k_heads: int, num_v_heads: int, head_dim: int = 128):
        self.indptr = _indptr(q_indptr)
        self.c = SdGdnShape(len(self.indptr) - 1, ctypes.cast(self.indptr, ctypes.POINTER(ctypes.c_int)),
                            int(num_k_heads), int(num_v_heads), int(head_dim))

    @property
    def ref(self):
        return ctypes.byref(self.c)


def sd_gdn_tree_cache_size(shape: GdnShape) -> int:
    return int(load().sd_gdn_tree_cache_size(shape.ref))


def sd_gdn_conv_tree(q_indptr, x, weight, conv_state, parents, y, dev_status=None, stream=None) -> None:
    """x, y bf16 [sumN, C]; weight fp32 [C, 4]; conv_state bf16 [B, C, 3]."""
    ind = _indptr(q_indptr)
    _check(load().sd_gdn_conv_tree(len(ind) - 1, ind, int(x.shape[-1]), _ptr(x), _ptr(weight), _ptr(conv_state),
                                   _ptr(parents), _ptr(y), _ptr(dev_status), _stream(stream)),
           "sd_gdn_conv_tree")


def sd_gdn_tree(shape: GdnShape, q, k, v, g, beta, state, parents, out, tree_cache, dev_status=None,
                stream=None) -> None:
    cache_bytes = tree_cache.numel() * tree_cache.element_size()
    _check(load().sd_gdn_tree(shape.ref, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(parents),
                              _ptr(out), _ptr(tree_cache), cache_bytes, _ptr(dev_status), _stream(stream)),
           "sd_gdn_tree")


def sd_gdn_commit(shape: GdnShape, state_layers, tree_cache_layers, accept_len, path, conv_state_layers=None,
                  x_layers=None, max_path: int | None = None, dev_status=None, stream=None) -> None:
    n = len(state_layers)
    if len(tree_cache_layers) != n:
        raise ValueError("per-layer lists differ in length")
    channels = 0
    conv_arr = x_arr = None
    if conv_state_layers is not None:
        if len(conv_state_layers) != n or x_layers is None or len(x_layers) != n:
            raise ValueError("per-layer lists differ in length")
        channels = int(x_layers[0].shape[-1])
        conv_arr, x_arr = _ptr_array(conv_state_layers), _ptr_array(x_layers)
    if max_path is None:
        max_path = path.shape[-1]
    _check(load().sd_gdn_commit(shape.ref, n, _ptr_array(state_layers), _ptr_array(tree_cache_layers), channels,
                                conv_arr, x_arr, _ptr(accept_len), _ptr(path), int(max_path), _ptr(dev_status),
                                _stream(stream)),
           "sd_gdn_commit")


# ---------------------------------------------------------------- the 8-bit block-scaled cache (include/sd_kv8.h)
#
# These calls check types, shapes, layouts and devices here.  A call is a few microseconds of Python beside a few of
# GPU time at the smallest sizes, so the checks are plain comparisons and what they refuse is explained elsewhere.

def _refuse(t, what: str, dtype, shape, index: int):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: a tensor is needed, got {type(t).__name__}")
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: {dtype} {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{what} is on {t.device}, other tensors are not")
    raise ValueError(f"{what} must be contiguous" if t.dim() != 3 else f"{what}: the heads of a row must be contiguous")


def _tensor(t, what: str, dtype, shape, index: int) -> int:
    """Address of a dense tensor of this type and shape on device `index`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, what, dtype, shape, index)


def _rows(t, what: str, shape, index: int) -> tuple[int, int]:
    """Address and row stride (0: dense) of bf16 [rows, heads, dim]; the rows may lie apart, a row is dense.  Rows that
    share memory (a tensor expanded along them has stride 0, which the C ABI takes for dense) are refused."""
    if t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == index:
        if t.is_contiguous():
            return t.data_ptr(), 0
        if t.stride(2) == 1 and (shape[1] == 1 or t.stride(1) == shape[2]):
            if shape[0] <= 1:
                return t.data_ptr(), 0
            if t.stride(0) < shape[1] * shape[2]:
                raise ValueError(f"{what}: the rows overlap (row stride {t.stride(0)}, a row has {shape[1] * shape[2]} values)")
            return t.data_ptr(), t.stride(0)
    _refuse(t, what, torch.bfloat16, shape, index)


_array_types = {}


def _array(ctype, values):
    """A ctypes array; its type is made once per length (making one takes longer than a call)."""
    key = (ctype, len(values))
    kind = _array_types.get(key)
    if kind is None:
        kind = _array_types[key] = ctype * key[1]
    return kind(*values)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(call, what: str, args, index: int, stream) -> None:
    """call(*args, stream) with device `index` current; the default stream is the device's current one."""
    if index < 0:
        raise ValueError(f"{what}: the tensors must be on a CUDA device")
    if stream is not None:
        stream = stream if isinstance(stream, int) else stream.cuda_stream
    elif _raw_stream is not None:
        stream = _raw_stream(index)
    else:
        stream = torch.cuda.current_stream(index).cuda_stream
    if torch.cuda.current_device() == index:
        status = call(*args, stream)
    else:
        with torch.cuda.device(index):
            status = call(*args, stream)
    if status != SD_OK:
        raise SdError(status, what)


def _put_layers(ptrs, x, n: int, what: str, dtype, shape, nbytes: int, index: int) -> None:
    """Append the device addresses of n per-layer tensors (a list of them, or one tensor with a leading layer dimension)."""
    if isinstance(x, torch.Tensor):
        base = _tensor(x, what, dtype, (n, *shape), index)
        ptrs.extend(range(base, base + nbytes * n, nbytes) if nbytes else [base] * n)
    elif len(x) == n:
        ptrs.extend([_tensor(t, what, dtype, shape, index) for t in x])
    else:
        raise ValueError(f"{what}: {n} layers expected, got {len(x)}")


def _put_rows(ptrs, x, n: int, what: str, heads: int, dim: int, index: int) -> tuple[int, int]:
    """The same for per-layer bf16 [rows, heads, dim]; returns the layers' common row stride and row count."""
    if isinstance(x, torch.Tensor) and x.dim() == 4 and x.is_contiguous():
        rows = x.shape[1]
        _put_layers(ptrs, x, n, what, torch.bfloat16, (rows, heads, dim), 2 * rows * heads * dim, index)
        return 0, rows
    if len(x) != n:
        raise ValueError(f"{what}: {n} layers expected, got {len(x)}")
    rows = x[0].shape[0] if x[0].dim() else 0
    got = [_rows(t, what, (rows, heads, dim), index) for t in x]
    if any(s != got[0][1] for _, s in got):
        raise ValueError(f"{what}: the layers differ in row stride")
    ptrs.extend([a for a, _ in got])
    return got[0][1], rows


_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


def sd_pages_extend(ctx_lens, add_lens, page_table, held, new_held, free_list, free_count, new_free_count, slots,
                    rows=None, row_indptr=None, new_ctx_lens=None, q_indptr=None, path=None, dev_status=None,
                    stream=None) -> None:
    """Pages and slot map for the ``add_lens`` tokens that join every sequence; with ``path`` (and the host
    ``q_indptr``) the accepted nodes of sd_accept, whose ``accept_len`` is ``add_lens``."""
    dev = page_table.get_device()
    if page_table.dim() != 2 or slots.dim() != 1 or free_list.dim() != 1:
        raise ValueError("page_table is [batch, pages], slots and free_list are one-dimensional")
    table_shape = page_table.shape
    batch, max_pages = table_shape
    each, one, max_rows, pool = (batch,), (1,), slots.shape[0], free_list.shape[0]
    ind, path_at, max_path = None, None, 0
    if q_indptr is not None or path is not None:
        if q_indptr is not None:
            ind = _array(ctypes.c_int, q_indptr if isinstance(q_indptr, list) else np.asarray(q_indptr).tolist())
        if ind is not None and len(ind) != batch + 1:
            raise ValueError("q_indptr has one entry more than the page table has rows")
        if path is not None:
            max_path = path.shape[-1] if path.dim() else 0
            path_at = _tensor(path, "path", _I32, (batch, max_path), dev)
    args = (batch, max_pages, pool, _tensor(ctx_lens, "ctx_lens", _I32, each, dev),
            _tensor(add_lens, "add_lens", _I32, each, dev), ind, path_at, max_path,
            _tensor(page_table, "page_table", _I32, table_shape, dev), _tensor(held, "held", _I32, each, dev),
            _tensor(new_held, "new_held", _I32, each, dev), _tensor(free_list, "free_list", _I32, (pool,), dev),
            _tensor(free_count, "free_count", _I32, one, dev),
            _tensor(new_free_count, "new_free_count", _I32, one, dev), max_rows,
            _tensor(slots, "slots", _I32, (max_rows,), dev),
            None if rows is None else _tensor(rows, "rows", _I32, (max_rows,), dev),
            None if row_indptr is None else _tensor(row_indptr, "row_indptr", _I32, (batch + 1,), dev),
            None if new_ctx_lens is None else _tensor(new_ctx_lens, "new_ctx_lens", _I32, each, dev),
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, one, dev))
    _run(load().sd_pages_extend, "sd_pages_extend", args, dev, stream)


def sd_pages_release(keep_lens, page_table, held, new_held, free_list, free_count, new_free_count, dev_status=None,
                     stream=None) -> None:
    """Pages behind the first ``keep_lens`` tokens of every sequence back on the free list."""
    dev = page_table.get_device()
    if page_table.dim() != 2 or free_list.dim() != 1:
        raise ValueError("page_table is [batch, pages], free_list is one-dimensional")
    table_shape = page_table.shape
    batch, max_pages = table_shape
    each, one, pool = (batch,), (1,), free_list.shape[0]
    args = (batch, max_pages, pool, _tensor(keep_lens, "keep_lens", _I32, each, dev),
            _tensor(page_table, "page_table", _I32, table_shape, dev), _tensor(held, "held", _I32, each, dev),
            _tensor(new_held, "new_held", _I32, each, dev), _tensor(free_list, "free_list", _I32, (pool,), dev),
            _tensor(free_count, "free_count", _I32, one, dev),
            _tensor(new_free_count, "new_free_count", _I32, one, dev),
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, one, dev))
    _run(load().sd_pages_release, "sd_pages_release", args, dev, stream)


def sd_kv8_append(k_cache_layers, v_cache_layers, k_scale_layers, v_scale_layers, k_new_layers, v_new_layers, slots,
                  rows=None, dev_status=None, stream=None) -> None:
    """bf16 rows quantised into the caches of every layer at the slots of a slot map (sd_pages_extend).

    Per layer (lists, or tensors with a leading layer dimension): codes uint8 [pool, heads, 16, dim], scales fp32
    [pool, heads], new rows bf16 [rows, heads, dim] (rows may lie apart, not overlap)."""
    dev, first = slots.get_device(), k_cache_layers
    if not isinstance(first, torch.Tensor):
        if not first:
            raise ValueError("no layers")
        n, cache = len(first), tuple(first[0].shape)
    else:
        shape = first.shape
        n, cache = (shape[0], shape[1:]) if shape else (0, ())
    if len(cache) != 4 or slots.dim() != 1:
        raise ValueError("a layer's cache is [pool, heads, 16, dim], slots is one-dimensional")
    pool, heads, page, dim = cache
    max_rows = slots.shape[0]
    block, codes = (pool, heads), pool * heads * page * dim
    ptrs = array("Q")      # the six arrays of n addresses, one behind the other
    _put_layers(ptrs, first, n, "k_cache", _U8, cache, codes, dev)
    _put_layers(ptrs, v_cache_layers, n, "v_cache", _U8, cache, codes, dev)
    _put_layers(ptrs, k_scale_layers, n, "k_scales", _F32, block, 4 * pool * heads, dev)
    _put_layers(ptrs, v_scale_layers, n, "v_scales", _F32, block, 4 * pool * heads, dev)
    stride, src = _put_rows(ptrs, k_new_layers, n, "k_new", heads, dim, dev)
    if (stride, src) != _put_rows(ptrs, v_new_layers, n, "v_new", heads, dim, dev):
        raise ValueError("k_new and v_new differ in rows or row stride")
    at, step = ptrs.buffer_info()[0], 8 * n
    args = (n, heads, dim, page, pool, at, at + step, at + 2 * step, at + 3 * step, at + 4 * step, at + 5 * step, stride,
            src,
            _tensor(slots, "slots", _I32, (max_rows,), dev),
            None if rows is None else _tensor(rows, "rows", _I32, (max_rows,), dev), max_rows,
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, (1,), dev))
    _run(load().sd_kv8_append, "sd_kv8_append", args, dev, stream)


def sd_kv8_attn_workspace_size(shape: Shape) -> int:
    return int(load().sd_kv8_attn_workspace_size(shape.ref))


def sd_kv8_attn(shape: Shape, q, k_cache, v_cache, k_scales, v_scales, k_new, v_new, page_table, ctx_lens, parents,
                out, lse=None, scale: float = 0.0, softcap: float = 0.0, slopes=None, workspace=None, dev_status=None,
                stream=None) -> None:
    """sd_verify_attn over the block-scaled cache; ``softcap`` and ``slopes`` (fp32 [query heads]) as in sd_kv8_opts.
    q, k_new and v_new may have rows that lie apart (slices of a fused projection), not rows that overlap."""
    dev = q.get_device()
    q_shape, kv_shape, cache, block, table, batch, n = shape.dims
    q_at, qs = _rows(q, "q", q_shape, dev)
    k_at, ks = _rows(k_new, "k_new", kv_shape, dev)
    v_at, vs = _rows(v_new, "v_new", kv_shape, dev)
    opts = None
    if scale or softcap or qs or ks or vs or slopes is not None:
        opts = ctypes.byref(SdKv8Opts(scale, softcap, None if slopes is None else
                                      _tensor(slopes, "slopes", _F32, (q_shape[1],), dev), qs, ks, vs))
    ws_at, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws_at = _tensor(workspace, "workspace", workspace.dtype, workspace.shape, dev)
    args = (shape.ref, opts, q_at, _tensor(k_cache, "k_cache", _U8, cache, dev),
            _tensor(v_cache, "v_cache", _U8, cache, dev), _tensor(k_scales, "k_scales", _F32, block, dev),
            _tensor(v_scales, "v_scales", _F32, block, dev), k_at, v_at,
            _tensor(page_table, "page_table", _I32, table, dev), _tensor(ctx_lens, "ctx_lens", _I32, batch, dev),
            _tensor(parents, "parents", _I32, n, dev), _tensor(out, "out", torch.bfloat16, q_shape, dev),
            None if lse is None else _tensor(lse, "lse", _F32, q_shape[:2], dev), ws_at, ws_bytes,
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, (1,), dev))
    _run(load().sd_kv8_attn, "sd_kv8_attn", args, dev, stream)


# ---------------------------------------------------------------- the 4-bit cache (include/sd_kv4.h)

def kv4_cache_shape(num_pool_pages: int, num_kv_heads: int, head_dim: int) -> tuple[int, int, int, int]:
    """Shape of one layer's 4-bit cache (uint8)."""
    return int(num_pool_pages), int(num_kv_heads), 2, 9 * int(head_dim)


def _kv4_layers(cache_layers):
    """(layers, one layer's shape) of a list of caches or a tensor with a leading layer dimension."""
    if isinstance(cache_layers, torch.Tensor):
        shape = cache_layers.shape
        n, cache = (shape[0], tuple(shape[1:])) if shape else (0, ())
    else:
        if not cache_layers:
            raise ValueError("no layers")
        n, cache = len(cache_layers), tuple(cache_layers[0].shape)
    if len(cache) != 4 or cache[2] != 2 or cache[3] % 9:
        raise ValueError("a layer's 4-bit cache is uint8 [pool, heads, 2, 9 * dim]")
    return n, cache


def _kv4_rows(cache_layers, k_layers, v_layers, slots, names):
    """Checked arguments of sd_kv4_append and sd_kv4_read: sizes, addresses (the array keeps them alive), stride, rows."""
    dev = slots.get_device()
    if slots.dim() != 1:
        raise ValueError("slots is one-dimensional")
    try:
        # the usual case, a tensor each with a leading layer dimension: in one go (the checks are half of a small call)
        n, pool, heads, two, width = cache_layers.shape
        shape = k_layers.shape
        each, row = pool * heads * 2 * width, 2 * shape[1] * shape[2] * shape[3]
        if len(shape) == 4 and each and row and n and two == 2 and width == 9 * shape[3] and shape[2] == heads and shape[0] == n \
                and v_layers.shape == shape and cache_layers.dtype is _U8 \
                and k_layers.dtype is torch.bfloat16 and v_layers.dtype is torch.bfloat16 \
                and cache_layers.get_device() == dev and k_layers.get_device() == dev and v_layers.get_device() == dev \
                and cache_layers.is_contiguous() and k_layers.is_contiguous() and v_layers.is_contiguous():
            at = cache_layers.data_ptr()
            ptrs = array("Q", range(at, at + each * n, each))
            at = k_layers.data_ptr()
            ptrs.extend(range(at, at + row * n, row))
            at = v_layers.data_ptr()
            ptrs.extend(range(at, at + row * n, row))
            at = ptrs.buffer_info()[0]
            return ptrs, (n, heads, shape[3], 16, pool, at, at + 8 * n, at + 16 * n, 0), shape[1], dev
    except (AttributeError, ValueError, IndexError):
        pass
    n, cache = _kv4_layers(cache_layers)
    pool, heads, dim = cache[0], cache[1], cache[3] // 9
    ptrs = array("Q")      # the three arrays of n addresses, one behind the other
    _put_layers(ptrs, cache_layers, n, "cache", _U8, cache, pool * heads * 18 * dim, dev)
    stride, rows = _put_rows(ptrs, k_layers, n, names[0], heads, dim, dev)
    if (stride, rows) != _put_rows(ptrs, v_layers, n, names[1], heads, dim, dev):
        raise ValueError(f"{names[0]} and {names[1]} differ in rows or row stride")
    at, step = ptrs.buffer_info()[0], 8 * n
    return ptrs, (n, heads, dim, 16, pool, at, at + step, at + 2 * step, stride), rows, dev


def sd_kv4_append(cache_layers, k_new_layers, v_new_layers, slots, rows=None, dev_status=None, stream=None) -> None:
    """bf16 rows quantised into the 4-bit caches of every layer at the slots of a slot map (sd_pages_extend).

    Per layer (lists, or tensors with a leading layer dimension): cache uint8 [pool, heads, 2, 9 * dim], new rows bf16
    [rows, heads, dim] (rows may lie apart, not overlap)."""
    ptrs, head, src, dev = _kv4_rows(cache_layers, k_new_layers, v_new_layers, slots, ("k_new", "v_new"))
    max_rows = slots.shape[0]
    args = (*head, src, _tensor(slots, "slots", _I32, (max_rows,), dev),
            None if rows is None else _tensor(rows, "rows", _I32, (max_rows,), dev), max_rows,
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, (1,), dev))
    _run(load().sd_kv4_append, "sd_kv4_append", args, dev, stream)


def sd_kv4_read(cache_layers, slots, k_out_layers, v_out_layers, dev_status=None, stream=None) -> None:
    """The values at these slots of the 4-bit caches of every layer, as bf16 rows [len(slots), heads, dim] (rows of slot
    -1 stay as they are)."""
    ptrs, head, rows, dev = _kv4_rows(cache_layers, k_out_layers, v_out_layers, slots, ("k_out", "v_out"))
    max_rows = slots.shape[0]
    if rows != max_rows:
        raise ValueError(f"k_out has {rows} rows, slots {max_rows}")
    args = (*head, _tensor(slots, "slots", _I32, (max_rows,), dev), max_rows,
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, (1,), dev))
    _run(load().sd_kv4_read, "sd_kv4_read", args, dev, stream)


def sd_kv4_attn_workspace_size(shape: Shape) -> int:
    return int(load().sd_kv4_attn_workspace_size(shape.ref))


def sd_kv4_attn(shape: Shape, q, cache, k_new, v_new, page_table, ctx_lens, parents, out, lse=None, scale: float = 0.0,
                softcap: float = 0.0, slopes=None, workspace=None, dev_status=None, stream=None) -> None:
    """sd_verify_attn over the 4-bit cache; ``softcap`` and ``slopes`` (fp32 [query heads]) as in sd_kv8_opts.
    q, k_new and v_new may have rows that lie apart (slices of a fused projection), not rows that overlap."""
    dev = q.get_device()
    q_shape, kv_shape, codes, _, table, batch, n = shape.dims
    q_at, qs = _rows(q, "q", q_shape, dev)
    k_at, ks = _rows(k_new, "k_new", kv_shape, dev)
    v_at, vs = _rows(v_new, "v_new", kv_shape, dev)
    opts = None
    if scale or softcap or qs or ks or vs or slopes is not None:
        opts = ctypes.byref(SdKv8Opts(scale, softcap, None if slopes is None else
                                      _tensor(slopes, "slopes", _F32, (q_shape[1],), dev), qs, ks, vs))
    ws_at, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws_at = _tensor(workspace, "workspace", workspace.dtype, workspace.shape, dev)
    args = (shape.ref, opts, q_at, _tensor(cache, "cache", _U8, (codes[0], codes[1], 2, 9 * codes[3]), dev), k_at, v_at,
            _tensor(page_table, "page_table", _I32, table, dev), _tensor(ctx_lens, "ctx_lens", _I32, batch, dev),
            _tensor(parents, "parents", _I32, n, dev), _tensor(out, "out", torch.bfloat16, q_shape, dev),
            None if lse is None else _tensor(lse, "lse", _F32, q_shape[:2], dev), ws_at, ws_bytes,
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, (1,), dev))
    _run(load().sd_kv4_attn, "sd_kv4_attn", args, dev, stream)


# ---------------------------------------------------------------- rotation and append (include/sd_rope.h)

def sd_rope_append(table, positions, q=None, k=None, v=None, q_out=None, k_out=None, k_cache=None, v_cache=None,
                   slots=None, interleaved: bool = False, dev_status=None, stream=None) -> None:
    """q and k rows turned to their positions into ``q_out`` and ``k_out`` (which may be q and k), and with ``v``, the
    bf16 caches [pool, heads, 16, dim] and ``slots`` also appended there.  ``table`` fp32 [positions, rot_dim]:
    cosines, then sines (step.rope_table).  q, k, v and the outputs may have rows that lie apart."""
    dev = table.get_device()
    if table.dim() != 2 or positions.dim() != 1:
        raise ValueError("table is [positions, rot_dim], positions is one-dimensional")
    table_len, rot = table.shape
    rows = positions.shape[0]
    some = q if q is not None else k
    if some is None or some.dim() != 3:
        raise ValueError("q and k are [rows, heads, dim]; one of them is needed")
    dim = some.shape[2]
    q_at = k_at = v_at = qo_at = ko_at = kc_at = vc_at = slots_at = None
    qs = ks = vs = qos = kos = hq = hkv = pool = 0
    if q is not None:
        shape = (rows, q.shape[1], dim)
        hq = shape[1]
        q_at, qs = _rows(q, "q", shape, dev)
    if q_out is not None:
        qo_at, qos = _rows(q_out, "q_out", (rows, hq, dim), dev)
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k is [rows, heads, dim]")
        shape = (rows, k.shape[1], dim)
        hkv = shape[1]
        k_at, ks = _rows(k, "k", shape, dev)
    if k_out is not None:
        ko_at, kos = _rows(k_out, "k_out", (rows, hkv, dim), dev)
    if v is not None:
        v_at, vs = _rows(v, "v", (rows, hkv, dim), dev)
    if k_cache is not None:
        pool = k_cache.shape[0] if k_cache.dim() else 0
        kc_at = _tensor(k_cache, "k_cache", torch.bfloat16, (pool, hkv, 16, dim), dev)
    if v_cache is not None:
        vc_at = _tensor(v_cache, "v_cache", torch.bfloat16, (pool, hkv, 16, dim), dev)
    if slots is not None:
        slots_at = _tensor(slots, "slots", _I32, (rows,), dev)
    shape = SdRopeShape(rows, hq, hkv, dim, rot, 1 if interleaved else 0, table_len, 16, pool, qs, ks, vs, qos, kos)
    args = (ctypes.byref(shape), _tensor(table, "table", _F32, (table_len, rot), dev),
            _tensor(positions, "positions", _I32, (rows,), dev), q_at, k_at, v_at, qo_at, ko_at, kc_at, vc_at, slots_at,
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, (1,), dev))
    _run(load().sd_rope_append, "sd_rope_append", args, dev, stream)


# ---------------------------------------------------------------- log probabilities (include/sd_logprobs.h)

_LOGITS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def sd_logprobs_workspace_size(num_rows: int, vocab: int, top: int) -> int:
    """Bytes for a call of these sizes; fewer rows may need more (they are cut into more pieces)."""
    return int(load().sd_logprobs_workspace_size(int(num_rows), int(vocab), int(top)))


def sd_logprobs(logits, tokens=None, logprobs=None, top_ids=None, top_logprobs=None, entropy=None, lse=None,
                temperature: float = 1.0, workspace=None, dev_status=None, stream=None) -> None:
    """Log probabilities of ``tokens`` int32 [rows, given], the largest logits' ids and log probabilities [rows, top],
    entropy and log-sum-exp [rows] of logits [rows, vocab] (fp32, bf16 or fp16; the rows may lie apart)."""
    dev = logits.get_device()
    dtype = _LOGITS.get(logits.dtype)
    if dtype is None or logits.dim() != 2:
        raise ValueError("logits are fp32, bf16 or fp16 [rows, vocab]")
    rows, vocab = logits.shape
    stride = 0
    if not logits.is_contiguous():
        stride = logits.stride(0) if rows > 1 else 0
        if (vocab > 1 and logits.stride(1) != 1) or (rows > 1 and stride < vocab):
            raise ValueError("logits: a row must be contiguous, and rows must not overlap")
    given, top = 0, 0
    if tokens is not None:
        given = tokens.shape[-1] if tokens.dim() else 0
        tokens = _tensor(tokens, "tokens", _I32, (rows, given), dev)
    if logprobs is not None:
        logprobs = _tensor(logprobs, "logprobs", _F32, (rows, given), dev)
    if top_ids is not None:
        top = top_ids.shape[-1] if top_ids.dim() else 0
        top_ids = _tensor(top_ids, "top_ids", _I32, (rows, top), dev)
    if top_logprobs is not None:
        top_logprobs = _tensor(top_logprobs, "top_logprobs", _F32, (rows, top), dev)
    ws_at, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws_at = _tensor(workspace, "workspace", workspace.dtype, workspace.shape, dev)
    args = (rows, vocab, dtype, logits.data_ptr(), stride, temperature, given, tokens or None, logprobs or None, top,
            top_ids or None, top_logprobs or None,
            None if entropy is None else _tensor(entropy, "entropy", _F32, (rows,), dev),
            None if lse is None else _tensor(lse, "lse", _F32, (rows,), dev), ws_at, ws_bytes,
            None if dev_status is None else _tensor(dev_status, "dev_status", _I32, (1,), dev))
    _run(load().sd_logprobs, "sd_logprobs", args, dev, stream)
