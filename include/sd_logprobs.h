/*
 * sd_logprobs.h — C ABI of the log probabilities of given tokens, with entropy
 * and top alternatives (sm_103a): what a server returns beside the tokens that
 * sd_accept or sd_sample_accept emit, from the same logits rows.
 *
 * Conventions are those of sd_verify.h: device pointers owned by the caller, no
 * allocation, no synchronisation, everything asynchronous on `stream` and
 * capturable into a CUDA graph; host-checkable errors are returned before any
 * launch; device-only problems OR a bit into *dev_status (nullable).
 */
#ifndef SD_LOGPROBS_H_
#define SD_LOGPROBS_H_

#include <stddef.h>

#include "sd_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SD_LOGITS_F32 0
#define SD_LOGITS_BF16 1
#define SD_LOGITS_F16 2

#define SD_LOGPROBS_MAX_TOP 32
#define SD_LOGPROBS_MAX_GIVEN 64
#define SD_LOGPROBS_MAX_VOCAB (1 << 24)

/* Bytes of workspace sd_logprobs needs for a call of these sizes (0 on bad arguments, and where rows are not cut into pieces).
 * Few rows are cut into more pieces than many, so fewer rows may need more: one workspace for calls of several sizes is as
 * large as the largest need among them. */
size_t sd_logprobs_workspace_size(int num_rows, int vocab, int top);

/*
 * sd_logprobs — per logits row x, with z = x / temperature:
 *   lse      = log(sum_v exp(z_v))
 *   logprobs = z_t - lse for each of the row's given tokens t; a token outside
 *              [0, vocab) (-1 as padding) has probability 0: -infinity
 *   entropy  = lse - sum_v p_v z_v with p = exp(z - lse), in nats; terms of
 *              p = 0 count 0
 *   top_ids, top_logprobs = the `top` largest logits, largest first, ties by
 *              the smaller index (-0.0 == +0.0), and their log-probabilities
 * Sums are fp32.  A logit of -infinity is a token that cannot come.  A row of
 * nothing else has lse = -infinity, entropy 0, log-probabilities -infinity and
 * the first `top` indices.  A NaN or a +infinity in a row sets
 * SD_DEV_NAN_LOGITS: its lse, entropy and log-probabilities are then NaN, its
 * top_ids -1.
 *
 *   num_rows     >= 0;  vocab  1..SD_LOGPROBS_MAX_VOCAB
 *   dtype        SD_LOGITS_F32, _BF16 or _F16
 *   logits       [num_rows][vocab], aligned to its type; rows row_stride elements apart (0: dense; else >= vocab)
 *   temperature  host float > 0 (finite, with a finite reciprocal)
 *   given        0..SD_LOGPROBS_MAX_GIVEN tokens a row;  tokens int32 [num_rows][given], logprobs fp32 the same
 *                (written); both NULL with given 0
 *   top          0..min(vocab, SD_LOGPROBS_MAX_TOP);  top_ids int32 [num_rows][top], top_logprobs fp32 the same
 *                (written); both NULL with top 0
 *   entropy, lse fp32 [num_rows] or NULL (written)
 *   workspace    >= sd_logprobs_workspace_size bytes, 16-byte aligned; two calls that may run at the same time need
 *                one each
 * No output may overlap an input or another output.
 */
sd_status sd_logprobs(int num_rows, int vocab, int dtype, const void* logits, long long row_stride, float temperature,
                      int given, const int* tokens, float* logprobs, int top, int* top_ids, float* top_logprobs,
                      float* entropy, float* lse, void* workspace, size_t ws_bytes, int* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SD_LOGPROBS_H_ */
