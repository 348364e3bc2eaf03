// C-ABI entry points of the 8-bit block-scaled cache (include/sd_kv8.h):
// host-side argument checks and launches.  Nothing here allocates device
// memory or synchronises.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

using namespace sdv;

namespace {

sd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SD_OK : SD_ERR_CUDA; }
bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// int32 and fp32 arrays start on 4 bytes.
template <typename... T>
bool words(const T*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ... | uintptr_t{0}) & 3u) == 0;
}

// Whether one of the arrays that a call writes is one that it reads, or written twice (nulls are no arrays).
template <int W, int R>
bool aliased(const int* const (&written)[W], const int* const (&read)[R]) {
  for (int i = 0; i < W; ++i) {
    if (written[i] == nullptr) continue;
    for (int j = 0; j < i; ++j)
      if (written[j] == written[i]) return true;
    for (const int* r : read)
      if (r == written[i]) return true;
  }
  return false;
}

sd_status check_pages(int batch, int max_pages, int pool) {
  if (batch < 1 || max_pages < 1 || pool < 1) return SD_ERR_INVALID_ARG;
  if (batch > kMaxBatch || (long long)max_pages * kPage > (1LL << 30) || (long long)pool * kPage > INT_MAX)
    return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

sd_status check_heads(int heads, int dim, int page_size) {
  if (heads < 1 || dim < 1 || page_size < 1) return SD_ERR_INVALID_ARG;
  if (heads > kMaxKvHeads || (dim != 128 && dim != 256) || page_size != kPage) return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

// A row stride: dense, or at least a row and a whole number of 16-byte pieces.
bool stride_ok(long long stride, long long row, long long* use) {
  *use = stride == 0 ? row : stride;
  return *use >= row && *use % 8 == 0 && *use <= (1LL << 40);
}

sd_status check_kv8_shape(const sd_shape* s, BatchDesc* bd) {
  if (s == nullptr) return SD_ERR_INVALID_ARG;
  sd_status st = check_heads(s->num_kv_heads, s->head_dim, s->page_size);
  if (st != SD_OK) return st;
  if (s->num_q_heads < 1 || s->num_q_heads % s->num_kv_heads != 0) return SD_ERR_INVALID_ARG;
  if (s->num_q_heads / s->num_kv_heads > kMaxGroup) return SD_ERR_UNSUPPORTED;
  if (s->num_splits < 0 || s->window < 0) return SD_ERR_INVALID_ARG;
  if (s->num_splits != 0) return SD_ERR_UNSUPPORTED;
  st = check_pages(s->batch < 1 ? 1 : s->batch, s->max_pages_per_seq, s->num_pool_pages);
  if (st != SD_OK) return st;
  // a half page of one head is a tensor-map coordinate; tiles are counted in 32 bits over the whole batch
  if ((long long)s->num_pool_pages * s->num_kv_heads * 2 > INT_MAX) return SD_ERR_UNSUPPORTED;
  const long long tiles = ((long long)s->max_pages_per_seq * kPage + kTileTokens - 1) / kTileTokens + 1;
  if (tiles * s->num_q_heads * (s->batch < 1 ? 1 : s->batch) > INT_MAX / 2) return SD_ERR_UNSUPPORTED;
  return fill_batch(s->batch, s->q_indptr_h, bd);
}

}  // namespace

extern "C" {

sd_status sd_pages_extend(int batch, int max_pages_per_seq, int num_pool_pages, const int* ctx_lens,
                          const int* add_lens, const int* q_indptr_h, const int* path, int max_path,
                          int* page_table, const int* held, int* new_held, const int* free_list,
                          const int* free_count, int* new_free_count, int max_rows, int* slots, int* rows,
                          int* row_indptr, int* new_ctx_lens, int* dev_status, void* stream) {
  const sd_status st = check_pages(batch, max_pages_per_seq, num_pool_pages);
  if (st != SD_OK) return st;
  if (!ctx_lens || !add_lens || !page_table || !held || !new_held || !free_list || !free_count || !new_free_count ||
      max_rows < 0 || (max_rows > 0 && !slots))
    return SD_ERR_INVALID_ARG;
  if (!words(ctx_lens, add_lens, path, page_table, held, new_held, free_list, free_count, new_free_count, slots, rows,
             row_indptr, new_ctx_lens, dev_status))
    return SD_ERR_INVALID_ARG;
  if ((q_indptr_h == nullptr) != (path == nullptr) || (path != nullptr && max_path < 1)) return SD_ERR_INVALID_ARG;
  if (aliased({page_table, new_held, new_free_count, slots, rows, row_indptr, new_ctx_lens, dev_status},
              {ctx_lens, add_lens, held, free_count, free_list, path}))
    return SD_ERR_INVALID_ARG;
  BatchDesc bd;
  std::memset(&bd, 0, sizeof(bd));
  if (q_indptr_h != nullptr) {
    const sd_status sb = fill_batch(batch, q_indptr_h, &bd);
    if (sb != SD_OK) return sb;
  }
  PagesParams p;
  std::memset(&p, 0, sizeof(p));
  p.ctx_lens = ctx_lens;
  p.add_lens = add_lens;
  p.path = path;
  p.page_table = page_table;
  p.held = held;
  p.new_held = new_held;
  p.free_list = free_list;
  p.free_count = free_count;
  p.new_free_count = new_free_count;
  p.slots = slots;
  p.rows = rows;
  p.row_indptr = row_indptr;
  p.new_ctx_lens = new_ctx_lens;
  p.dev_status = dev_status;
  p.batch = batch;
  p.max_pages = max_pages_per_seq;
  p.num_pool_pages = num_pool_pages;
  p.max_path = max_path;
  p.max_rows = max_rows;
  p.vec = aligned(slots, 16) && aligned(rows, 16);
  return cuda_status(launch_pages_extend(p, bd, static_cast<cudaStream_t>(stream)));
}

sd_status sd_pages_release(int batch, int max_pages_per_seq, int num_pool_pages, const int* keep_lens,
                           const int* page_table, const int* held, int* new_held, int* free_list,
                           const int* free_count, int* new_free_count, int* dev_status, void* stream) {
  const sd_status st = check_pages(batch, max_pages_per_seq, num_pool_pages);
  if (st != SD_OK) return st;
  if (!keep_lens || !page_table || !held || !new_held || !free_list || !free_count || !new_free_count)
    return SD_ERR_INVALID_ARG;
  if (!words(keep_lens, page_table, held, new_held, free_list, free_count, new_free_count, dev_status))
    return SD_ERR_INVALID_ARG;
  if (aliased({new_held, new_free_count, free_list, dev_status}, {keep_lens, held, free_count, page_table}))
    return SD_ERR_INVALID_ARG;
  PagesParams p;
  std::memset(&p, 0, sizeof(p));
  p.ctx_lens = keep_lens;
  p.page_table = const_cast<int*>(page_table);   // read only
  p.held = held;
  p.new_held = new_held;
  p.free_list_out = free_list;
  p.free_count = free_count;
  p.new_free_count = new_free_count;
  p.dev_status = dev_status;
  p.batch = batch;
  p.max_pages = max_pages_per_seq;
  p.num_pool_pages = num_pool_pages;
  return cuda_status(launch_pages_release(p, static_cast<cudaStream_t>(stream)));
}

sd_status sd_kv8_append(int num_layers, int num_kv_heads, int head_dim, int page_size, int num_pool_pages,
                        void* const* k_cache_layers, void* const* v_cache_layers, float* const* k_scale_layers,
                        float* const* v_scale_layers, const void* const* k_new_layers,
                        const void* const* v_new_layers, long long new_stride, int num_src_rows,
                        const int* slots, const int* rows, int max_rows, int* dev_status, void* stream) {
  sd_status st = check_heads(num_kv_heads, head_dim, page_size);
  if (st != SD_OK) return st;
  st = check_pages(1, 1, num_pool_pages);
  if (st != SD_OK) return st;
  if (num_layers < 1 || max_rows < 0 || num_src_rows < 0) return SD_ERR_INVALID_ARG;
  if (num_layers > kMaxLayers) return SD_ERR_UNSUPPORTED;
  if (!k_cache_layers || !v_cache_layers || !k_scale_layers || !v_scale_layers || !k_new_layers || !v_new_layers ||
      (max_rows > 0 && !slots))
    return SD_ERR_INVALID_ARG;
  if (!words(slots, rows, dev_status)) return SD_ERR_INVALID_ARG;
  Kv8AppendParams p;
  std::memset(&p, 0, sizeof(p));
  if (!stride_ok(new_stride, (long long)num_kv_heads * head_dim, &p.new_stride)) return SD_ERR_INVALID_ARG;
  for (int l = 0; l < num_layers; ++l) {
    const void* all[6] = {k_cache_layers[l], v_cache_layers[l], k_new_layers[l], v_new_layers[l],
                          k_scale_layers[l], v_scale_layers[l]};
    for (int i = 0; i < 6; ++i)
      if (all[i] == nullptr || !aligned(all[i], i < 4 ? 16 : 4)) return SD_ERR_INVALID_ARG;
    p.k_cache[l] = static_cast<uint8_t*>(k_cache_layers[l]);
    p.v_cache[l] = static_cast<uint8_t*>(v_cache_layers[l]);
    p.k_scale[l] = k_scale_layers[l];
    p.v_scale[l] = v_scale_layers[l];
    p.k_new[l] = static_cast<const __nv_bfloat16*>(k_new_layers[l]);
    p.v_new[l] = static_cast<const __nv_bfloat16*>(v_new_layers[l]);
  }
  p.slots = slots;
  p.rows = rows;
  p.dev_status = dev_status;
  p.num_layers = num_layers;
  p.heads = num_kv_heads;
  p.dim = head_dim;
  p.num_pool_pages = num_pool_pages;
  p.num_src_rows = num_src_rows;
  p.max_rows = max_rows;
  return cuda_status(launch_kv8_append(p, static_cast<cudaStream_t>(stream)));
}

size_t sd_kv8_attn_workspace_size(const sd_shape* shape) {
  BatchDesc bd;
  if (check_kv8_shape(shape, &bd) != SD_OK) return 0;
  return kv8_attn_workspace(shape->num_q_heads, shape->num_kv_heads, shape->head_dim, bd);
}

sd_status sd_kv8_attn(const sd_shape* shape, const sd_kv8_opts* opts, const void* q, const void* k_cache,
                      const void* v_cache, const float* k_scales, const float* v_scales, const void* k_new,
                      const void* v_new, const int* page_table, const int* ctx_lens, const int* parents,
                      void* out, float* lse, void* workspace, size_t ws_bytes, int* dev_status, void* stream) {
  BatchDesc bd;
  const sd_status st = check_kv8_shape(shape, &bd);
  if (st != SD_OK) return st;
  if (!q || !k_cache || !v_cache || !k_scales || !v_scales || !k_new || !v_new || !page_table || !ctx_lens ||
      !parents || !out)
    return SD_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_new, 16) ||
      !aligned(v_new, 16) || !aligned(out, 16) || !aligned(workspace, 16) || out == q)
    return SD_ERR_INVALID_ARG;
  if (!words(k_scales, v_scales, page_table, ctx_lens, parents, lse, dev_status)) return SD_ERR_INVALID_ARG;
  Kv8AttnParams p;
  std::memset(&p, 0, sizeof(p));
  const long long q_row = (long long)shape->num_q_heads * shape->head_dim;
  const long long kv_row = (long long)shape->num_kv_heads * shape->head_dim;
  sd_kv8_opts o;
  std::memset(&o, 0, sizeof(o));
  if (opts != nullptr) o = *opts;
  if (!std::isfinite(o.scale) || o.scale < 0.f || !std::isfinite(o.softcap) || o.softcap < 0.f ||
      !aligned(o.slopes, 4) || !stride_ok(o.q_stride, q_row, &p.q_stride) ||
      !stride_ok(o.k_stride, kv_row, &p.k_stride) || !stride_ok(o.v_stride, kv_row, &p.v_stride))
    return SD_ERR_INVALID_ARG;
  if (o.softcap > SD_KV8_MAX_SOFTCAP) return SD_ERR_UNSUPPORTED;
  const size_t need = kv8_attn_workspace(shape->num_q_heads, shape->num_kv_heads, shape->head_dim, bd);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return SD_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.page_table = page_table;
  p.ctx_lens = ctx_lens;
  p.parents = parents;
  p.slopes = o.slopes;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.dev_status = dev_status;
  p.scale = o.scale > 0.f ? o.scale : 1.0f / std::sqrt((float)shape->head_dim);
  // a smaller cap leaves scores of 2^-20 at most either way, and the factors of the capped form out of range
  p.softcap = o.softcap > 0.f ? std::fmax(o.softcap, 0x1p-20f) : 0.f;
  p.cap_exp = o.softcap > 0.f ? 2.0f / p.softcap : 0.f;
  p.hq = shape->num_q_heads;
  p.hkv = shape->num_kv_heads;
  p.group = p.hq / p.hkv;
  p.dim = shape->head_dim;
  p.max_pages = shape->max_pages_per_seq;
  p.num_pool_pages = shape->num_pool_pages;
  p.window = shape->window;
  p.workspace = workspace;
  return cuda_status(launch_kv8_attn(p, bd, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
