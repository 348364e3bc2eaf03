// C-ABI entry points of the 4-bit cache (include/sd_kv4.h): host-side argument
// checks and launches.  Nothing here allocates device memory or synchronises.
#include <climits>

#include "api_checks.cuh"

using namespace sdv;

namespace {

// Arguments that the append and the read share, into the parameter block (rows and source rows apart).
sd_status fill_rows(int num_layers, int heads, int dim, int page_size, int pool, const void* const* cache_layers,
                    const void* const* k_layers, const void* const* v_layers, long long stride, const int* slots,
                    int max_rows, int* dev_status, Kv4RowsParams* p) {
  sd_status st = check_heads(heads, dim, page_size);
  if (st != SD_OK) return st;
  st = check_pages(1, 1, pool);
  if (st != SD_OK) return st;
  if (num_layers < 1 || max_rows < 0) return SD_ERR_INVALID_ARG;
  if (num_layers > kMaxLayers) return SD_ERR_UNSUPPORTED;
  if (!cache_layers || !k_layers || !v_layers || (max_rows > 0 && !slots)) return SD_ERR_INVALID_ARG;
  if (!words(slots, dev_status)) return SD_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  if (!stride_ok(stride, (long long)heads * dim, &p->stride)) return SD_ERR_INVALID_ARG;
  for (int l = 0; l < num_layers; ++l) {
    if (!cache_layers[l] || (max_rows > 0 && (!k_layers[l] || !v_layers[l])) || !aligned(cache_layers[l], 16) || !aligned(k_layers[l], 16) ||
        !aligned(v_layers[l], 16))
      return SD_ERR_INVALID_ARG;
    p->cache[l] = static_cast<uint8_t*>(const_cast<void*>(cache_layers[l]));
    p->k_rows[l] = static_cast<__nv_bfloat16*>(const_cast<void*>(k_layers[l]));
    p->v_rows[l] = static_cast<__nv_bfloat16*>(const_cast<void*>(v_layers[l]));
  }
  p->slots = slots;
  p->dev_status = dev_status;
  p->num_layers = num_layers;
  p->heads = heads;
  p->num_pool_pages = pool;
  p->max_rows = max_rows;
  return SD_OK;
}

}  // namespace

extern "C" {

sd_status sd_kv4_append(int num_layers, int num_kv_heads, int head_dim, int page_size, int num_pool_pages,
                        void* const* cache_layers, const void* const* k_new_layers, const void* const* v_new_layers,
                        long long new_stride, int num_src_rows, const int* slots, const int* rows, int max_rows,
                        int* dev_status, void* stream) {
  Kv4RowsParams p;
  const sd_status st = fill_rows(num_layers, num_kv_heads, head_dim, page_size, num_pool_pages, cache_layers,
                                 k_new_layers, v_new_layers, new_stride, slots, max_rows, dev_status, &p);
  if (st != SD_OK) return st;
  if (num_src_rows < 0 || !words(rows)) return SD_ERR_INVALID_ARG;
  for (int l = 1; l < num_layers; ++l)       // a cache given for two layers would have two writers
    for (int k = 0; k < l; ++k)
      if (p.cache[k] == p.cache[l]) return SD_ERR_INVALID_ARG;
  p.rows = rows;
  p.num_src_rows = num_src_rows;
  return cuda_status(launch_kv4_append(p, head_dim, static_cast<cudaStream_t>(stream)));
}

sd_status sd_kv4_read(int num_layers, int num_kv_heads, int head_dim, int page_size, int num_pool_pages,
                      const void* const* cache_layers, void* const* k_out_layers, void* const* v_out_layers,
                      long long out_stride, const int* slots, int max_rows, int* dev_status, void* stream) {
  Kv4RowsParams p;
  const sd_status st = fill_rows(num_layers, num_kv_heads, head_dim, page_size, num_pool_pages, cache_layers,
                                 k_out_layers, v_out_layers, out_stride, slots, max_rows, dev_status, &p);
  if (st != SD_OK) return st;
  for (int l = 0; l < num_layers; ++l) {     // an array given for two outputs, or a cache for one
    if (max_rows == 0) break;
    if (p.k_rows[l] == p.v_rows[l]) return SD_ERR_INVALID_ARG;
    for (int k = 0; k < num_layers; ++k) {
      const void* cache = p.cache[k];
      if (cache == p.k_rows[l] || cache == p.v_rows[l]) return SD_ERR_INVALID_ARG;
      if (k < l && (p.k_rows[k] == p.k_rows[l] || p.v_rows[k] == p.v_rows[l] || p.k_rows[k] == p.v_rows[l] ||
                    p.v_rows[k] == p.k_rows[l]))
        return SD_ERR_INVALID_ARG;
    }
  }
  return cuda_status(launch_kv4_read(p, head_dim, static_cast<cudaStream_t>(stream)));
}

size_t sd_kv4_attn_workspace_size(const sd_shape* shape) {
  BatchDesc bd;
  if (check_kv_shape(shape, &bd) != SD_OK) return 0;
  return kv4_attn_workspace(shape->num_q_heads, shape->num_kv_heads, shape->head_dim, bd);
}

sd_status sd_kv4_attn(const sd_shape* shape, const sd_kv8_opts* opts, const void* q, const void* cache,
                      const void* k_new, const void* v_new, const int* page_table, const int* ctx_lens,
                      const int* parents, void* out, float* lse, void* workspace, size_t ws_bytes, int* dev_status,
                      void* stream) {
  BatchDesc bd;
  const sd_status st = check_kv_shape(shape, &bd);
  if (st != SD_OK) return st;
  if (!q || !cache || !k_new || !v_new || !page_table || !ctx_lens || !parents || !out) return SD_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16) || out == q)
    return SD_ERR_INVALID_ARG;
  if (!words(page_table, ctx_lens, parents, lse, dev_status)) return SD_ERR_INVALID_ARG;
  Kv4AttnParams p;
  std::memset(&p, 0, sizeof(p));
  const sd_status so = set_opts(shape, opts, &p);
  if (so != SD_OK) return so;
  const size_t need = kv4_attn_workspace(shape->num_q_heads, shape->num_kv_heads, shape->head_dim, bd);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return SD_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.page_table = page_table;
  p.ctx_lens = ctx_lens;
  p.parents = parents;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.dev_status = dev_status;
  p.hq = shape->num_q_heads;
  p.hkv = shape->num_kv_heads;
  p.group = p.hq / p.hkv;
  p.dim = shape->head_dim;
  p.max_pages = shape->max_pages_per_seq;
  p.num_pool_pages = shape->num_pool_pages;
  p.window = shape->window;
  p.workspace = workspace;
  return cuda_status(launch_kv4_attn(p, bd, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
