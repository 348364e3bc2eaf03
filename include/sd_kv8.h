/*
 * sd_kv8.h — C ABI of the 8-bit block-scaled K/V cache (sm_103a): its page
 * tables and slot maps, the quantising append, and the verify attention that
 * reads it.
 *
 * The cache of one layer.  Pages of 16 tokens come from one pool, as in
 * sd_verify.h; a page holds, for every KV head, 16 rows of e4m3 codes
 * (1 sign, 4 exponent bits with bias 7, 3 mantissa bits; subnormals m * 2^-9;
 * 0x7F / 0xFF are NaN; largest 448):
 *   K and V codes   uint8 [num_pool_pages][num_kv_heads][16][head_dim]
 *   K and V scales  fp32  [num_pool_pages][num_kv_heads]
 * A code stands for decode(code) * scale of its (page, KV head).  Where the
 * caches of sd_verify_attn_fp8 have one host scale per layer and tensor, chosen
 * before the data is known, these follow the data block by block.
 *
 * The usual step:
 *   sd_kv8_attn of every layer -> sd_accept -> sd_pages_extend (pages and slot
 *   map of the accepted path) -> sd_kv8_append of every layer in one launch.
 * A prompt takes sd_pages_extend without a path, then sd_kv8_append; a
 * sequence that ends or rolls back takes sd_pages_release.
 *
 * Conventions are those of sd_verify.h: device pointers owned by the caller, no
 * allocation, no synchronisation, everything asynchronous on `stream` and
 * capturable into a CUDA graph; host-checkable errors are returned before any
 * launch; device-only problems OR a bit into *dev_status (nullable).  bf16
 * tensors, codes and workspaces start on 16 bytes, int32 and fp32 arrays on 4.
 * Geometry here: 16-token pages; head_dim 128 or 256; num_kv_heads 1..64;
 * num_q_heads = G * num_kv_heads with G 1..16 (query head h reads KV head
 * h / G); N_b 1..64 nodes a sequence (1 = plain single-token decoding).
 */
#ifndef SD_KV8_H_
#define SD_KV8_H_

#include <stddef.h>

#include "sd_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of *dev_status. */
#define SD_DEV_NO_PAGES   128   /* sd_pages_extend: the free list is too short; nothing was changed */
#define SD_DEV_BAD_SCALE  256   /* a cache scale outside [2^-100, 2^100] (or NaN) was read */
#define SD_DEV_BAD_SLOT   512   /* a slot map names a slot or source row out of range, or breaks its order; or more
                                   rows than the map has room for */

#define SD_KV8_MIN_SCALE_EXP (-100)
#define SD_KV8_MAX_SCALE_EXP 100
#define SD_KV8_MAX_SOFTCAP 4096.0f

/*
 * sd_pages_extend — page-table entries and the slot map for the tokens that
 * join every sequence, from the free list, on the GPU.
 *
 * Sequence b holds its first held[b] page-table entries and has ctx_lens[b]
 * tokens; add_lens[b] >= 0 tokens join it at positions ctx .. ctx + add - 1.
 * It then needs need = max(held, ceil((ctx + add) / 16)) pages; entries
 * held .. need - 1 are taken from the top of the free list, sequence by
 * sequence:
 *   page_table[b][j] = free_list[free_count - 1 - (o_b + j - held[b])],
 * o_b being the number of pages that the sequences before b take.  The new
 * tokens are rows 0, 1, 2, ... in sequence order, position by position:
 *   slots[r]  = page_table[b][pos / 16] * 16 + pos % 16,
 *   rows[r]   = q_indptr_h[b] + path[b][i] for the i-th new token of b when a
 *               path is given (the accepted nodes of sd_accept, whose
 *               accept_len is add_lens), else r,
 *   row_indptr[b] = first row of b, row_indptr[B] = number of rows;
 * slots and rows behind the last row are -1 up to max_rows (sd_kv8_append
 * skips them).
 *
 * All or nothing: when a sequence's lengths are wrong (negative, beyond
 * max_pages_per_seq pages, ctx_lens not held: SD_DEV_BAD_CTX), the path is
 * (SD_DEV_BAD_ACCEPT), the rows exceed max_rows (SD_DEV_BAD_SLOT) or the free
 * list is too short (SD_DEV_NO_PAGES), then the page table stays as it was,
 * the new_* outputs repeat the old values, and every slot and row is -1.  A
 * page id out of [0, num_pool_pages) that a row lands on sets SD_DEV_BAD_PAGE;
 * that row's slot is -1.
 *
 *   batch, max_pages_per_seq, num_pool_pages   B 1..SD_MAX_BATCH; max_pages_per_seq * 16 <= 2^30,
 *                            num_pool_pages * 16 < 2^31
 *   ctx_lens, add_lens       int32 [B]
 *   q_indptr_h, path, max_path   host [B+1] and int32 [B][max_path], both or neither; max_path >= 1 with them
 *   page_table               int32 [B][max_pages_per_seq], entries [0, held) read, [held, need) written
 *   held, new_held           int32 [B]; free_list int32 [num_pool_pages], entries [0, *free_count) are free pages
 *   free_count, new_free_count   int32 [1]
 *   slots                    int32 [max_rows]; rows int32 [max_rows] or NULL; row_indptr int32 [B+1] or NULL
 *   new_ctx_lens             int32 [B] or NULL: ctx + add
 * No output may alias an input (nor new_ctx_lens the ctx_lens) or another
 * output, dev_status among them; the page table is updated in place.  Pages
 * shared between sequences are not tracked.
 */
sd_status sd_pages_extend(int batch, int max_pages_per_seq, int num_pool_pages, const int* ctx_lens,
                          const int* add_lens, const int* q_indptr_h, const int* path, int max_path,
                          int* page_table, const int* held, int* new_held, const int* free_list,
                          const int* free_count, int* new_free_count, int max_rows, int* slots, int* rows,
                          int* row_indptr, int* new_ctx_lens, int* dev_status, void* stream);

/*
 * sd_pages_release — pages behind the first keep_lens[b] tokens of every
 * sequence go back on the free list (keep 0: the sequence ends; keep >= what
 * it holds: nothing happens to it).
 *
 * keep = min(held, ceil(keep_lens / 16)) pages stay; entries keep .. held - 1
 * are pushed sequence by sequence: free_list[free_count + o_b + j - keep] =
 * page_table[b][j], o_b being the pages released before b.  new_held[b] = keep;
 * *new_free_count = *free_count + all of them.  The page table is not written.
 * All or nothing as above: a negative keep_lens or held outside [0,
 * max_pages_per_seq] (SD_DEV_BAD_CTX), or more pages than free_list has room
 * for (SD_DEV_BAD_PAGE), changes nothing and repeats the old values.  A
 * released id out of [0, num_pool_pages) sets SD_DEV_BAD_PAGE and is pushed as
 * it is.  No output may alias an input or another output; free_list is updated
 * in place behind entry *free_count - 1.
 */
sd_status sd_pages_release(int batch, int max_pages_per_seq, int num_pool_pages, const int* keep_lens,
                           const int* page_table, const int* held, int* new_held, int* free_list,
                           const int* free_count, int* new_free_count, int* dev_status, void* stream);

/*
 * sd_kv8_append — bf16 K/V rows quantised into the cache at the slots of a
 * slot map, for every layer, in one launch.
 *
 * Row r goes to slot slots[r] (page slots[r] / 16, token slots[r] % 16) and
 * comes from source row rows[r] (r itself without rows); slots[r] = -1 is
 * skipped.  The rows of one page are consecutive in the map, in rising
 * order without gaps, as sd_pages_extend writes them (an order broken inside
 * a page sets SD_DEV_BAD_SLOT and the group of rows is skipped; a page that
 * comes back later in the map is not noticed: its content is then
 * unspecified).  Per (layer, K or V, page, KV head), with f the page's first
 * new token and amax the largest finite magnitude of the new values:
 *   s(amax) = 2^e, the smallest with amax <= 448 * 2^e, e clamped to
 *             [-100, 100] (an all-zero block takes 2^-100);
 *   f == 0: the page begins here, scale = s(amax);
 *   f > 0:  tokens 0 .. f-1 are valid; scale = max(old scale, s(amax)), and
 *           where it grew the old codes become e4m3(decode(code) * old / scale)
 *           (exact between powers of two down to e4m3's subnormals);
 *   new code = e4m3(x / scale): nearest, ties to the even code; finite values
 *           beyond 448 * scale and infinities saturate; NaN gives a NaN code.
 * Tokens behind the new rows of a page are left as they were.  An old scale
 * outside [2^-100, 2^100] sets SD_DEV_BAD_SCALE and the (page, head) is
 * skipped.
 *
 *   num_layers                 1..SD_MAX_LAYERS
 *   k_cache_layers .. v_new_layers   HOST arrays of num_layers device pointers: codes (written), scales
 *                              (written), new rows bf16 [num_src_rows][num_kv_heads][head_dim]
 *   new_stride                 elements between source rows: 0 (dense) or a multiple of 8 of at least
 *                              num_kv_heads * head_dim (rows inside a fused projection)
 *   slots, rows                int32 [max_rows], rows nullable; max_rows >= 0
 */
sd_status sd_kv8_append(int num_layers, int num_kv_heads, int head_dim, int page_size, int num_pool_pages,
                        void* const* k_cache_layers, void* const* v_cache_layers, float* const* k_scale_layers,
                        float* const* v_scale_layers, const void* const* k_new_layers,
                        const void* const* v_new_layers, long long new_stride, int num_src_rows,
                        const int* slots, const int* rows, int max_rows, int* dev_status, void* stream);

/* How sd_kv8_attn turns a dot product into a score; NULL = {0, 0, NULL, 0, 0, 0}. */
typedef struct sd_kv8_opts {
  float scale;            /* multiplies q.k; 0 = 1 / sqrt(head_dim); else positive and finite */
  float softcap;          /* c > 0: score = c * tanh(score / c) (applied before the bias); 0 = none.  At most
                             SD_KV8_MAX_SOFTCAP, else SD_ERR_UNSUPPORTED: the capped score is off by some c * 2^-22 */
  const float* slopes;    /* device fp32 [num_q_heads] or NULL: score += slopes[h] * (key position - query position),
                             a bias that falls with distance for positive slopes */
  long long q_stride;     /* elements between rows of q: 0 (dense) or a multiple of 8, >= num_q_heads * head_dim */
  long long k_stride;     /* the same for k_new: 0, or a multiple of 8, >= num_kv_heads * head_dim */
  long long v_stride;     /* the same for v_new */
} sd_kv8_opts;

/* Bytes of workspace sd_kv8_attn needs for this shape (0 on a bad shape). */
size_t sd_kv8_attn_workspace_size(const sd_shape* shape);

/*
 * sd_kv8_attn — sd_verify_attn over the block-scaled cache: tree/causal-masked
 * grouped-query attention of one layer, down to single-token decoding (N_b = 1).
 *
 * For sequence b, node j (position L_b + depth(j)) and query head h, the
 * output is softmax attention of q[j][h] over the keys of KV head h / G: the
 * L_b context tokens of the cache, then the draft nodes on j's root path
 * (bf16, from k_new / v_new, at their own positions).  Scores are formed as
 * sd_kv8_opts says; with shape->window = W > 0 node j sees keys at positions
 * > L_b + depth(j) - W only.
 *
 *   shape       geometry as above; window as in sd_verify.h; num_splits must be 0 (the split over
 *               the SMs is planned on the device from ctx_lens; else SD_ERR_UNSUPPORTED);
 *               ctx_stable is accepted and has no effect
 *   q           bf16 [sumN][num_q_heads][head_dim]
 *   k_cache, v_cache, k_scales, v_scales   one layer's cache (read only)
 *   k_new, v_new  bf16 [sumN][num_kv_heads][head_dim]
 *   page_table, ctx_lens, parents   as for sd_verify_attn
 *   out         bf16 [sumN][num_q_heads][head_dim] (written, dense)
 *   lse         fp32 [sumN][num_q_heads] or NULL: natural log of the sum of exp(scores)
 *   workspace   >= sd_kv8_attn_workspace_size(shape) bytes.  Its contents need not be kept between calls; two calls
 *               that may run at the same time need one each.
 *
 * Numerics: scores, softmax statistics, sums and the partial outputs of split
 * sequences are fp32.  The products take 8-bit operands: the cache's codes as
 * they lie; a query (one node's, of one head) as two e4m3 terms (off by at most
 * 2^-17 of its own amax); a draft key or value as two e4m3 terms (2^-17 of its
 * row's amax where that is above 448 * 2^-100; magnitudes beyond 448 * 2^100
 * saturate, as they would in the cache); a softmax weight times its token's V
 * scale as an e4m3 term and an e5m2 rest.  That product is off by at most 2^-7
 * of itself; below 2^-9 of the largest such product that its CTA has met in the
 * column by up to a quarter of itself, up or down by the token's place in its
 * 128-token tile, so that many alike are right in the mean; and below 2^-20
 * (2^-22 over more than 8192 tokens of a CTA, 2^-24 over 32768) it no longer
 * reaches the output.  So where tokens share the weight but their blocks' V
 * scales lie further apart than 2^9, the values of the small blocks lose bits,
 * and beyond 2^20 they are lost, in dims that the large blocks leave at zero
 * too.  The sum of weights is not rounded.
 * Outputs are typically within 0.002 of their size, against 0.0017 for the
 * rounding to bf16 alone.  A page id out of range sets SD_DEV_BAD_PAGE and its
 * tokens count as zeros; a scale out of range sets SD_DEV_BAD_SCALE and is
 * clamped.  Codes at masked positions (behind L_b, before a window, on other
 * branches) never reach an output, whatever they hold.  A NaN or an infinity in
 * a q row makes that row's output NaN, one in a k_new or v_new row the outputs
 * of the nodes that see it.
 */
sd_status sd_kv8_attn(const sd_shape* shape, const sd_kv8_opts* opts, const void* q, const void* k_cache,
                      const void* v_cache, const float* k_scales, const float* v_scales, const void* k_new,
                      const void* v_new, const int* page_table, const int* ctx_lens, const int* parents,
                      void* out, float* lse, void* workspace, size_t ws_bytes, int* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SD_KV8_H_ */
