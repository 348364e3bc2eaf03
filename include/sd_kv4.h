/*
 * sd_kv4.h — C ABI of the 4-bit K/V cache (sm_103a): the quantising append,
 * rows read back out of it, and the verify attention on the codes.
 *
 * «如何在单张 RTX 3090 上让 Qwen3.5-27B token 生成速度提升 6 倍» (24 GB 显存上的 128K
 * 上下文) keeps the cache in 4-bit blocks of 32 values with one scale each, so
 * that 128K tokens of context fit beside the weights.  This is such a cache
 * for the paged pool of sd_verify.h: a value is
 *   (c - 8) * s,   c a 4-bit code 0..15, s the scale of its token, KV head and
 *                  block of 32 dims,
 * 4.5 bits a value.  s is a bf16 with 5 significant bits (the 3 lowest bits of
 * the number are zero; they are ignored where they are not), so (c - 8) * s is
 * exactly a bf16 value: the attention's operands are the cache's values
 * themselves.  Scales are at most SD_KV4_MAX_SCALE in magnitude.
 *
 * One (page, KV head) of one layer, 18 * head_dim consecutive bytes in
 *   cache   uint8 [num_pool_pages][num_kv_heads][2][9 * head_dim]:
 * the K record, then the V record.  Eight codes make one 32-bit word (little
 * endian), code e of the eight at bit 16 * (e % 2) + 4 * (e / 2).
 *   K   words [head_dim / 32][16 tokens][4]   of 8 consecutive dims of a token
 *       scales bf16 [16 tokens][head_dim / 32]
 *   V   words [head_dim][2]                   of 8 consecutive tokens of a dim
 *       scales bf16 [head_dim / 32][16 tokens]
 *
 * The usual step is that of sd_kv8.h: sd_kv4_attn of every layer -> sd_accept
 * -> sd_pages_extend (pages and slot map of the accepted path) ->
 * sd_kv4_append of every layer in one launch.
 *
 * Conventions are those of sd_verify.h: device pointers owned by the caller, no
 * allocation, no synchronisation, everything asynchronous on `stream` and
 * capturable into a CUDA graph; host-checkable errors are returned before any
 * launch; device-only problems OR a bit into *dev_status (nullable).  bf16
 * tensors, caches and workspaces start on 16 bytes, int32 and fp32 arrays on 4.
 * Geometry: 16-token pages; head_dim 128 or 256; num_kv_heads 1..64;
 * num_q_heads = G * num_kv_heads with G 1..16 (query head h reads KV head
 * h / G); N_b 1..64 nodes a sequence (1 = plain single-token decoding).
 */
#ifndef SD_KV4_H_
#define SD_KV4_H_

#include <stddef.h>

#include "sd_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SD_KV4_MAX_SCALE 0x1.5p123f   /* 1.3125 * 2^123 */

/* Further bits of *dev_status (SD_DEV_BAD_SCALE and SD_DEV_BAD_SLOT are those of sd_kv8.h). */
#define SD_DEV_NOT_FINITE 1024   /* sd_kv4_append met a NaN or an infinity, for which 4 bits have no code */

/*
 * sd_kv4_append — bf16 K/V rows quantised into the cache at the slots of a
 * slot map, for every layer, in one launch.
 *
 * Row r goes to slot slots[r] (page slots[r] / 16, token slots[r] % 16) and
 * comes from source row rows[r] (r itself without rows); slots[r] = -1 is
 * skipped.  The rows of one page are consecutive in the map, in rising
 * order without gaps, as sd_pages_extend writes them (an order broken inside
 * a page sets SD_DEV_BAD_SLOT and the group of rows is skipped; a page that
 * comes back later in the map is not noticed: its content is then
 * unspecified).  Per row, KV head and block of 32 dims:
 *   m = the finite value largest in magnitude (the first of them),
 *   s = m / -8 rounded to 5 significant bits (ties to even; at most
 *       SD_KV4_MAX_SCALE in magnitude), 0 where |m| < 2^-100,
 *   c = rint(x / s) + 8, ties to even, kept within 0..15; 8 (the value 0)
 *       where s = 0.
 * So m itself is held to half a unit of 5 bits, every other value within
 * |s| / 2, except that what is nearest to +8 s is held as 7 s (and that
 * magnitudes beyond 8 SD_KV4_MAX_SCALE = 1.12e38 saturate).  Infinities are
 * held as the end of the block's range on their side (as 0 where no finite value
 * of the block reaches 2^-100, whose scale is 0), NaN as 0; both set
 * SD_DEV_NOT_FINITE.  Tokens of a page that get no row are left as they were.
 *
 *   num_layers                 1..SD_MAX_LAYERS
 *   cache_layers               HOST array of num_layers device pointers (written)
 *   k_new_layers, v_new_layers HOST arrays of num_layers device pointers, bf16 [num_src_rows][num_kv_heads][head_dim]
 *   new_stride                 elements between source rows: 0 (dense) or a multiple of 8 of at least
 *                              num_kv_heads * head_dim (rows inside a fused projection)
 *   slots, rows                int32 [max_rows], rows nullable; max_rows >= 0
 */
sd_status sd_kv4_append(int num_layers, int num_kv_heads, int head_dim, int page_size, int num_pool_pages,
                        void* const* cache_layers, const void* const* k_new_layers, const void* const* v_new_layers,
                        long long new_stride, int num_src_rows, const int* slots, const int* rows, int max_rows,
                        int* dev_status, void* stream);

/*
 * sd_kv4_read — rows of the cache as bf16, for every layer, in one launch (a
 * sequence that moves to another cache, or what an append has stored).
 *
 * Row r of k_out and v_out becomes the values at slot slots[r], exactly;
 * slots[r] = -1 leaves the row as it was.  Slots may come in any order and
 * more than once (in rising order a page is read once for its 16 tokens).  A
 * slot out of the pool sets SD_DEV_BAD_SLOT and leaves the row; a scale beyond
 * SD_KV4_MAX_SCALE (infinities and NaN too) sets SD_DEV_BAD_SCALE and counts as 0.
 *
 *   k_out_layers, v_out_layers HOST arrays of num_layers device pointers, bf16 [max_rows][num_kv_heads][head_dim]
 *                              (written); no two of them, nor a cache, may overlap
 *   out_stride                 elements between their rows, as new_stride above
 *   slots                      int32 [max_rows]
 */
sd_status sd_kv4_read(int num_layers, int num_kv_heads, int head_dim, int page_size, int num_pool_pages,
                      const void* const* cache_layers, void* const* k_out_layers, void* const* v_out_layers,
                      long long out_stride, const int* slots, int max_rows, int* dev_status, void* stream);

/* Bytes of workspace sd_kv4_attn needs for this shape (0 on a bad shape). */
size_t sd_kv4_attn_workspace_size(const sd_shape* shape);

/*
 * sd_kv4_attn — sd_verify_attn over the 4-bit cache: tree/causal-masked
 * grouped-query attention of one layer, down to single-token decoding (N_b = 1).
 *
 * For sequence b, node j (position L_b + depth(j)) and query head h, the
 * output is softmax attention of q[j][h] over the keys of KV head h / G: the
 * L_b context tokens of the cache, then the draft nodes on j's root path
 * (bf16, from k_new / v_new, at their own positions).  Scores are formed as
 * sd_kv8_opts says (opts NULL: scale 1 / sqrt(head_dim), no cap, no bias);
 * with shape->window = W > 0 node j sees keys at positions > L_b + depth(j) - W
 * only.
 *
 *   shape       geometry as above; window as in sd_verify.h; num_splits must be 0 (the split over
 *               the SMs is planned on the device from ctx_lens; else SD_ERR_UNSUPPORTED);
 *               ctx_stable is accepted and has no effect
 *   q           bf16 [sumN][num_q_heads][head_dim]
 *   cache       one layer's cache (read only)
 *   k_new, v_new  bf16 [sumN][num_kv_heads][head_dim]
 *   page_table, ctx_lens, parents   as for sd_verify_attn
 *   out         bf16 [sumN][num_q_heads][head_dim] (written, dense); must not overlap q
 *   lse         fp32 [sumN][num_q_heads] or NULL: natural log of the sum of exp(scores)
 *   workspace   >= sd_kv4_attn_workspace_size(shape) bytes.  Its contents need not be kept between calls; two calls
 *               that may run at the same time need one each.
 *
 * Numerics: keys, values and queries enter the products as they are (bf16);
 * softmax weights are rounded to bf16 (by at most 2^-8 of themselves), their sum is not;
 * scores, statistics, sums and the partial outputs of split sequences are fp32
 * (a score beyond its range, 3.4e38, makes its row NaN).  The sum of weighted values
 * runs in the tensor core, which cuts off towards zero: over n keys in one CTA it is
 * off by up to n * 2^-27 of the sum of weight times |v| (values of one sign by 0.0007
 * of themselves over 131072 keys, by 0.006 over 2^20).  Values are summed up before
 * they are divided by the sum of the weights, and a weight may come to 2^16 before
 * a row's reference moves: for a row of n keys (L_b + depth + 1) no sum passes
 * fp32's range while n times the largest |v| is below 2^112 = 5e33; beyond that
 * an output may be an infinity or NaN although the mean itself is not.
 * A page id out of range sets SD_DEV_BAD_PAGE and its tokens count as zeros; a
 * scale beyond SD_KV4_MAX_SCALE (infinities and NaN too) sets SD_DEV_BAD_SCALE
 * and counts as 0 (at tokens that no query sees it is not looked at).  What lies at masked
 * positions (behind L_b, before a window, on other branches) never reaches an
 * output.  A NaN or an infinity in a q row makes that row's output NaN, one in
 * a k_new or v_new row the outputs of the nodes that see it.
 */
sd_status sd_kv4_attn(const sd_shape* shape, const sd_kv8_opts* opts, const void* q, const void* cache,
                      const void* k_new, const void* v_new, const int* page_table, const int* ctx_lens,
                      const int* parents, void* out, float* lse, void* workspace, size_t ws_bytes, int* dev_status,
                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SD_KV4_H_ */
