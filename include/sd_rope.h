/*
 * sd_rope.h — C ABI of the rotating append (sm_103a): query and key rows
 * turned to their positions, and the keys and values appended to the paged
 * bf16 cache on the way.
 *
 * sd_verify_attn and its kind take q, k_new and v_new after the rotation, and
 * sd_kv_commit moves what a verify step accepted; this call is what comes
 * before them (draft rows rotated, nothing appended yet) and the way in for
 * rows that need no verification: a prompt, a plainly decoded token.
 *
 * Conventions are those of sd_verify.h: device pointers owned by the caller, no
 * allocation, no synchronisation, everything asynchronous on `stream` and
 * capturable into a CUDA graph; host-checkable errors are returned before the
 * launch; device-only problems OR a bit into *dev_status (nullable).
 */
#ifndef SD_ROPE_H_
#define SD_ROPE_H_

#include <stddef.h>

#include "sd_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of *dev_status. */
#define SD_DEV_BAD_POSITION 2048   /* sd_rope_append: a position outside [-1, table_len) */

#define SD_ROPE_MAX_DIM 512
#define SD_ROPE_MAX_HEADS 1024

/* Sizes and layout of one call.  All fields are host values. */
typedef struct sd_rope_shape {
  int num_rows;          /* rows of every tensor, >= 0 (0: nothing is done, and no pointer is looked at) */
  int num_q_heads;       /* 0..SD_ROPE_MAX_HEADS; 0: no queries */
  int num_kv_heads;      /* 0..SD_ROPE_MAX_HEADS; 0: no keys and values */
  int head_dim;          /* a multiple of 16, 16..SD_ROPE_MAX_DIM */
  int rot_dim;           /* the first rot_dim dims of a head turn: a multiple of 16, 16..head_dim */
  int interleaved;       /* 0: dim i turns with dim i + rot_dim / 2; 1: dim 2 i with dim 2 i + 1 */
  int table_len;         /* positions in the table, >= 1 */
  int page_size;         /* must be 16 */
  int num_pool_pages;    /* pages of the caches, >= 1 (with caches only) */
  long long q_stride;    /* elements between rows: 0 (dense) or a multiple of 8 of at least a row */
  long long k_stride;
  long long v_stride;
  long long q_out_stride;
  long long k_out_stride;
} sd_rope_shape;

/*
 * sd_rope_append — for every row r at position p = positions[r]:
 *   pair i < rot_dim / 2 of every query and key head, with c = table[p][i] and
 *   s = table[p][rot_dim / 2 + i]:   y_a = x_a c - x_b s,   y_b = x_b c + x_a s
 *   (fp32, rounded once to bf16); dims from rot_dim on are copied;
 *   q_out[r] = the turned q[r];  k_out[r] = the turned k[r];
 *   slots[r] >= 0:  k_cache, v_cache at slot slots[r] (page slots[r] / 16,
 *   token slots[r] % 16) = the turned k[r], and v[r] as it is.
 * positions[r] = -1 is padding: nothing is written for the row.  A
 * position outside [-1, table_len) sets SD_DEV_BAD_POSITION and the row is
 * skipped; a slot below -1 or behind the pool sets SD_DEV_BAD_SLOT and the row
 * is not appended.  Rows that name the same slot leave values of either there.
 *
 *   table       fp32 [table_len][rot_dim]: cosines, then sines, of every position (angles of far positions lose
 *               their digits in fp32, so the table is best made in 64 bits), 16-byte aligned
 *   positions   int32 [num_rows]
 *   q, q_out    bf16 [num_rows][num_q_heads][head_dim], both or (num_q_heads 0) neither; 16-byte aligned
 *   k           bf16 [num_rows][num_kv_heads][head_dim], with k_out, the caches or both; NULL with num_kv_heads 0
 *   k_out       nullable
 *   v, k_cache, v_cache, slots   all or none: bf16 [num_rows][num_kv_heads][head_dim], bf16
 *               [num_pool_pages][num_kv_heads][16][head_dim] twice (written), int32 [num_rows]
 * q_out may be q, and k_out k, with the same stride (rotation in place); no
 * other output may overlap an input or another output.
 */
sd_status sd_rope_append(const sd_rope_shape* shape, const float* table, const int* positions, const void* q,
                         const void* k, const void* v, void* q_out, void* k_out, void* k_cache, void* v_cache,
                         const int* slots, int* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SD_ROPE_H_ */
