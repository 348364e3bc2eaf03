// Host checks shared by the C-ABI entry points of the quantised caches and of
// the calls beside them.  Internal to the library.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace sdv {
namespace {

inline sd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SD_OK : SD_ERR_CUDA; }
inline bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// int32 and fp32 arrays start on 4 bytes.
template <typename... T>
bool words(const T*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ... | uintptr_t{0}) & 3u) == 0;
}

inline sd_status check_pages(int batch, int max_pages, int pool) {
  if (batch < 1 || max_pages < 1 || pool < 1) return SD_ERR_INVALID_ARG;
  if (batch > kMaxBatch || (long long)max_pages * kPage > (1LL << 30) || (long long)pool * kPage > INT_MAX)
    return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

inline sd_status check_heads(int heads, int dim, int page_size) {
  if (heads < 1 || dim < 1 || page_size < 1) return SD_ERR_INVALID_ARG;
  if (heads > kMaxKvHeads || (dim != 128 && dim != 256) || page_size != kPage) return SD_ERR_UNSUPPORTED;
  return SD_OK;
}

// A row stride: dense, or at least a row and a whole number of 16-byte pieces.
inline bool stride_ok(long long stride, long long row, long long* use) {
  *use = stride == 0 ? row : stride;
  return *use >= row && *use % 8 == 0 && *use <= (1LL << 40);
}

inline sd_status check_kv_shape(const sd_shape* s, BatchDesc* bd) {
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

// The score options of an attention call, into its parameter block: strides, scale, cap, slopes.
template <typename P>
sd_status set_opts(const sd_shape* shape, const sd_kv8_opts* opts, P* p) {
  const long long q_row = (long long)shape->num_q_heads * shape->head_dim;
  const long long kv_row = (long long)shape->num_kv_heads * shape->head_dim;
  sd_kv8_opts o;
  std::memset(&o, 0, sizeof(o));
  if (opts != nullptr) o = *opts;
  if (!std::isfinite(o.scale) || o.scale < 0.f || !std::isfinite(o.softcap) || o.softcap < 0.f ||
      !aligned(o.slopes, 4) || !stride_ok(o.q_stride, q_row, &p->q_stride) ||
      !stride_ok(o.k_stride, kv_row, &p->k_stride) || !stride_ok(o.v_stride, kv_row, &p->v_stride))
    return SD_ERR_INVALID_ARG;
  if (o.softcap > SD_KV8_MAX_SOFTCAP) return SD_ERR_UNSUPPORTED;
  p->slopes = o.slopes;
  p->scale = o.scale > 0.f ? o.scale : 1.0f / std::sqrt((float)shape->head_dim);
  // a smaller cap leaves scores of 2^-20 at most either way, and the factors of the capped form out of range
  p->softcap = o.softcap > 0.f ? std::fmax(o.softcap, 0x1p-20f) : 0.f;
  p->cap_exp = o.softcap > 0.f ? 2.0f / p->softcap : 0.f;
  return SD_OK;
}

}  // namespace
}  // namespace sdv
