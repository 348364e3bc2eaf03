// C-ABI entry points beside the attention and the accept: the rotating append
// (include/sd_rope.h) and the log probabilities (include/sd_logprobs.h).
// Host-side argument checks and launches; nothing here allocates device
// memory or synchronises.
#include <climits>

#include "api_checks.cuh"

using namespace sdv;

extern "C" {

sd_status sd_rope_append(const sd_rope_shape* s, const float* table, const int* positions, const void* q,
                         const void* k, const void* v, void* q_out, void* k_out, void* k_cache, void* v_cache,
                         const int* slots, int* dev_status, void* stream) {
  if (s == nullptr) return SD_ERR_INVALID_ARG;
  if (s->num_rows < 0 || s->num_q_heads < 0 || s->num_kv_heads < 0 || s->head_dim < 1 || s->rot_dim < 1 ||
      s->table_len < 1 || s->interleaved < 0 || s->interleaved > 1)
    return SD_ERR_INVALID_ARG;
  if (s->num_q_heads > SD_ROPE_MAX_HEADS || s->num_kv_heads > SD_ROPE_MAX_HEADS || s->head_dim % 16 != 0 ||
      s->head_dim > SD_ROPE_MAX_DIM || s->rot_dim % 16 != 0)
    return SD_ERR_UNSUPPORTED;
  if (s->rot_dim > s->head_dim || s->num_q_heads + s->num_kv_heads == 0) return SD_ERR_INVALID_ARG;
  const bool has_q = s->num_q_heads > 0, has_k = s->num_kv_heads > 0, appends = k_cache != nullptr;
  if (s->num_rows == 0) return SD_OK;
  if (!table || !positions) return SD_ERR_INVALID_ARG;
  if ((q != nullptr) != has_q || (q_out != nullptr) != has_q || (k != nullptr) != has_k) return SD_ERR_INVALID_ARG;
  if ((v != nullptr) != appends || (v_cache != nullptr) != appends || (slots != nullptr) != appends)
    return SD_ERR_INVALID_ARG;
  // keys that go nowhere, or places without keys
  if (has_k ? (k_out == nullptr && !appends) : (k_out != nullptr || appends)) return SD_ERR_INVALID_ARG;
  if (appends) {
    if (s->page_size < 1 || s->num_pool_pages < 1) return SD_ERR_INVALID_ARG;
    if (s->page_size != kPage || (long long)s->num_pool_pages * kPage > INT_MAX) return SD_ERR_UNSUPPORTED;
  }
  for (const void* x : {static_cast<const void*>(table), q, k, v, static_cast<const void*>(q_out),
                        static_cast<const void*>(k_out), static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
    if (!aligned(x, 16)) return SD_ERR_INVALID_ARG;
  if (!words(positions, slots, dev_status)) return SD_ERR_INVALID_ARG;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  const long long q_row = (long long)s->num_q_heads * s->head_dim, kv_row = (long long)s->num_kv_heads * s->head_dim;
  if (!stride_ok(s->q_stride, q_row, &p.q_stride) || !stride_ok(s->k_stride, kv_row, &p.k_stride) ||
      !stride_ok(s->v_stride, kv_row, &p.v_stride) || !stride_ok(s->q_out_stride, q_row, &p.q_out_stride) ||
      !stride_ok(s->k_out_stride, kv_row, &p.k_out_stride))
    return SD_ERR_INVALID_ARG;
  // in place means row by row
  if ((has_q && q_out == q && p.q_out_stride != p.q_stride) || (k_out != nullptr && k_out == k && p.k_out_stride != p.k_stride))
    return SD_ERR_INVALID_ARG;
  // an array given for two outputs, or an input for another's output
  const void* outs[4] = {q_out, k_out, k_cache, v_cache};
  for (int i = 0; i < 4; ++i) {
    if (outs[i] == nullptr) continue;
    for (int j = 0; j < i; ++j)
      if (outs[j] == outs[i]) return SD_ERR_INVALID_ARG;
    if ((i != 0 && outs[i] == q) || (i != 1 && outs[i] == k) || outs[i] == v) return SD_ERR_INVALID_ARG;
  }
  p.table = table;
  p.positions = positions;
  p.slots = slots;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  p.dev_status = dev_status;
  p.num_rows = s->num_rows;
  p.hq = s->num_q_heads;
  p.hkv = s->num_kv_heads;
  p.dim = s->head_dim;
  p.rot_dim = s->rot_dim;
  p.interleaved = s->interleaved;
  p.table_len = s->table_len;
  p.num_pool_pages = s->num_pool_pages;
  return cuda_status(launch_rope_append(p, static_cast<cudaStream_t>(stream)));
}

size_t sd_logprobs_workspace_size(int num_rows, int vocab, int top) {
  if (num_rows < 0 || vocab < 1 || vocab > SD_LOGPROBS_MAX_VOCAB || top < 0 || top > SD_LOGPROBS_MAX_TOP || top > vocab)
    return 0;
  return logprobs_workspace(num_rows, vocab, top);
}

sd_status sd_logprobs(int num_rows, int vocab, int dtype, const void* logits, long long row_stride, float temperature,
                      int given, const int* tokens, float* logprobs, int top, int* top_ids, float* top_logprobs,
                      float* entropy, float* lse, void* workspace, size_t ws_bytes, int* dev_status, void* stream) {
  if (num_rows < 0 || vocab < 1 || dtype < SD_LOGITS_F32 || dtype > SD_LOGITS_F16 || given < 0 || top < 0 || top > vocab)
    return SD_ERR_INVALID_ARG;
  if (vocab > SD_LOGPROBS_MAX_VOCAB || given > SD_LOGPROBS_MAX_GIVEN || top > SD_LOGPROBS_MAX_TOP)
    return SD_ERR_UNSUPPORTED;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.0f / temperature)) return SD_ERR_INVALID_ARG;
  const bool rows = num_rows > 0;
  if ((rows && logits == nullptr) || !aligned(logits, dtype == SD_LOGITS_F32 ? 4 : 2)) return SD_ERR_INVALID_ARG;
  if (row_stride != 0 && (row_stride < vocab || row_stride > (1LL << 40))) return SD_ERR_INVALID_ARG;
  if (rows && ((tokens != nullptr) != (given > 0) || (logprobs != nullptr) != (given > 0) ||
               (top_ids != nullptr) != (top > 0) || (top_logprobs != nullptr) != (top > 0)))
    return SD_ERR_INVALID_ARG;
  if (!words(tokens, logprobs, top_ids, top_logprobs, entropy, lse, dev_status) || !aligned(workspace, 16))
    return SD_ERR_INVALID_ARG;
  const void* outs[5] = {logprobs, top_ids, top_logprobs, entropy, lse};
  for (int i = 0; i < 5; ++i) {
    if (outs[i] == nullptr) continue;
    if (outs[i] == logits || outs[i] == tokens) return SD_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[j] == outs[i]) return SD_ERR_INVALID_ARG;
  }
  const size_t need = logprobs_workspace(num_rows, vocab, top);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return SD_ERR_WORKSPACE;
  LogprobsParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.row_stride = row_stride == 0 ? vocab : row_stride;
  p.tokens = tokens;
  p.logprobs = logprobs;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  p.entropy = entropy;
  p.lse = lse;
  p.dev_status = dev_status;
  p.inv_t = 1.0f / temperature;
  p.num_rows = num_rows;
  p.vocab = vocab;
  p.dtype = dtype;
  p.given = given;
  p.top = top;
  return cuda_status(launch_logprobs(p, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
