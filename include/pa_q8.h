/*
 * pa_q8.h -- C ABI of the cache in 8 bits: new rows stored with a scale for
 * each block and KV head, read back, and attended to, whole or over blocks
 * that a cheap score selects.
 *
 * The cache (row-major, device memory):
 *   k_cache, v_cache [num_blocks][BLOCK][KV][D] int8 codes in [-127, 127]
 *   k_scale, v_scale [num_blocks][KV] float32
 *   bounds           [num_blocks][KV][2][D] int8: for each channel the lowest
 *                    and the highest code of the block's keys (only for
 *                    pa_q8_select)
 * Token i of sequence b is row i % BLOCK of block p = block_table[b][i /
 * BLOCK]; its key of KV head h is k_scale[p][h] * k_cache[p][i % BLOCK][h][:],
 * its value likewise.  D is 64 or 128, BLOCK 8, 16, 32 or 64; the dtype of
 * rows outside the cache is PA_F32, PA_F16 or PA_BF16.
 *
 * Every call is asynchronous on `stream`; the library keeps nothing.  Each
 * returns PA_OK or, before anything is launched, a PA_ERR_* code of
 * pa_decode.h:
 *   PA_ERR_NULL_POINTER  a needed pointer is NULL
 *   PA_ERR_BAD_DIMS      a size < 1 (B, N: < 0), H % KV != 0, max_blocks *
 *                        BLOCK >= 2^30, num_blocks * BLOCK >= 2^31, an output
 *                        that overlaps an input or another output
 *   PA_ERR_UNSUPPORTED   D, BLOCK or dtype outside the built set, B > 4096,
 *                        KV > 1024, and the limits of each call
 *   PA_ERR_ALIGNMENT     caches, bounds or rows not 16-byte aligned, another
 *                        tensor not 4-byte aligned, a stride not a multiple of
 *                        16 bytes or negative
 *   PA_ERR_WORKSPACE     (pa_q8_decode) too small or not 256-byte aligned
 * Device conditions are OR-ed into *status (device int32, may be NULL):
 *   PA_STATUS_BAD_LENGTH a length outside [0, max_blocks * BLOCK] or a count
 *                        outside its range (clamped)
 *   PA_STATUS_BAD_BLOCK  a table entry outside the pool, a selected block
 *                        outside the sequence: not read
 *   PA_STATUS_BAD_SLOT   pa_q8_append: a row that the table has no block for:
 *                        not stored
 *   PA_STATUS_NOT_FINITE pa_q8_append: an infinity or a NaN among the rows
 */
#ifndef PA_Q8_H
#define PA_Q8_H

#include <stddef.h>
#include <stdint.h>

#include "pa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PA_Q8_MIN_SCALE 1.262177448353619e-29f /* 2^-96 */

/*
 * Stores counts[b] new rows (counts NULL: N) of every sequence behind its
 * seq_lens[b] tokens: token seq_lens[b] + j gets k_new[b][h][j], v_new[b][h][j].
 * For each block that gets rows, each KV head, keys and values apart:
 *
 *   a     = largest magnitude of the new rows' finite values
 *   scale = max(a / 127, 2^-96), and the block's earlier scale where it holds
 *           earlier tokens (of this sequence, below seq_lens[b])
 *   codes of the new rows: the integer nearest to x / scale (ties to even) in
 *           [-127, 127]; an infinity is +-127, a NaN 0
 *   codes of the earlier rows, where the scale grew: the integer nearest to
 *           code * earlier scale / scale (ties to even)
 *   bounds (if given): lowest and highest code by channel of the block's keys,
 *           the earlier rows' and the new ones'
 *
 * a / 127 is rounded to float32, the quotients are not: the codes are exact.
 * A value is off by at most half its block's scale at the time it is stored,
 * and by half of each larger scale that the block gets later.  Rows of the
 * block behind the new ones are left as they were.  Only the sequence's own
 * blocks may be written: a block that two sequences share must be full, and the
 * table has to hold the sequence's own block for every new row or an entry outside
 * the pool (behind pa_plan_blocks: seq_lens and counts are its kept and granted).
 *
 * k_new, v_new [B][KV][N][D] of dtype with strides {batch, head, row} in
 * elements; columns contiguous.  N at most PA_MAX_PREFILL.  The outputs
 * (caches, scales, bounds) may not overlap the inputs or each other.
 */
typedef struct pa_q8_append_opts {
    int max_blocks, num_blocks, dtype;
    long long k_strides[3], v_strides[3];
    const int32_t *counts; /* [B], or NULL */
    int8_t *bounds;        /* or NULL */
    int *status;
} pa_q8_append_opts;

int pa_q8_append(int8_t *k_cache, int8_t *v_cache, float *k_scale, float *v_scale,
                 const void *k_new, const void *v_new, const int32_t *block_table,
                 const int32_t *seq_lens, int B, int KV, int D, int N, int BLOCK,
                 const pa_q8_append_opts *opts, void *stream);

/*
 * Reads tokens starts[b] .. starts[b] + counts[b] - 1 (counts NULL: N) of every
 * sequence back: k_out[b][h][j], v_out[b][h][j] [B][KV][N][D] of dtype, the
 * product of code and scale in float32, rounded to the dtype.  Rows j >=
 * counts[b], and rows whose block is not in the pool, are left as they were.
 * A token beyond the table is not read (PA_STATUS_BAD_LENGTH).
 */
typedef struct pa_q8_read_opts {
    int max_blocks, num_blocks, dtype;
    const int32_t *counts; /* [B], or NULL */
    int *status;
} pa_q8_read_opts;

int pa_q8_read(const int8_t *k_cache, const int8_t *v_cache, const float *k_scale,
               const float *v_scale, const int32_t *block_table, const int32_t *starts,
               void *k_out, void *v_out, int B, int KV, int D, int N, int BLOCK,
               const pa_q8_read_opts *opts, void *stream);

/*
 * Blocks of every sequence and KV head that the step's queries look at most.
 * With nb = ceil(seq_lens[b] / BLOCK): all of them when nb <= budget; else the
 * first keep_first, the last keep_last, and of those between the budget -
 * keep_first - keep_last with the highest scores (equal scores: the lowest
 * block first).  selected[b][h][0 .. m-1] are their indices in the table row in
 * ascending order, m = counts[b][h] = min(nb, budget); -1 behind them.
 *
 * The score bounds the products of the quantised queries with the block's
 * quantised keys from above, in whole numbers (a real product may exceed it by
 * the row's rounding).  For each query row of the KV head (H / KV heads, NQ rows):
 *   step  = max(largest finite magnitude / 127, 2^-96), as in pa_q8_append
 *   c     = the row's codes by that step, as in pa_q8_append
 *   total = sum over d of max(c[d] * bounds[0][d], c[d] * bounds[1][d])
 *   score = (step * k_scale) * total, each product rounded to float32
 * and the block's score is the largest over the rows.  A NaN (of a k_scale
 * that is none) counts as lower than any other score.
 *
 * q [B][H][NQ][D] of dtype, contiguous; selected [B][KV][budget], counts
 * [B][KV] int32.  Limits: max_blocks <= 32768, NQ <= PA_MAX_NQ, H / KV * NQ <=
 * 1024, B * KV <= 32768, keep_first + keep_last <= budget (else
 * PA_ERR_BAD_DIMS).  budget may exceed max_blocks.  Table entries behind a
 * sequence's blocks may be read, and are not used.
 */
typedef struct pa_q8_select_opts {
    int max_blocks, num_blocks, dtype;
    int budget, keep_first, keep_last;
    int *status;
} pa_q8_select_opts;

int pa_q8_select(const void *q, const int8_t *bounds, const float *k_scale,
                 const int32_t *block_table, const int32_t *seq_lens, int32_t *selected,
                 int32_t *counts, int B, int H, int KV, int D, int NQ, int BLOCK,
                 const pa_q8_select_opts *opts, void *stream);

/*
 * Attention of the step's query rows over the cache: with n = seq_lens[b]
 * tokens in the cache, the NQ new ones among them (pa_q8_append has stored
 * them), row r of head h sees keys 0 .. n - NQ + r (causal) or 0 .. n - 1:
 *
 *   out[b][h][r] = sum_i softmax_i(scale * q[b][h][r] . key_i) * value_i
 *
 * A row that sees no key gives zeros.  With `selected` and `counts`
 * ([B][KV][budget], [B][KV] int32: pa_q8_select's, or a caller's own) only the
 * keys of blocks selected[b][h / (H / KV)][0 .. counts-1] are seen; an entry
 * outside [0, ceil(n / BLOCK)) is skipped (-1 silently), a block named twice
 * counts twice.
 *
 * Scores, softmax statistics and sums are float32.  Codes are exact in the
 * products; 16-bit queries enter them with their own digits (those below 2^-35
 * of the row's largest element are lost), float32 queries with 22 bits, weights with 22, and with 11 where q is bfloat16 and H / KV * NQ
 * > 8.  out is of q's dtype.
 *
 * Scales have to be finite, key scales below 2^114 and value scales at most 2^96;
 * one below 2^-96 (0 among them) counts as 2^-96.  Value scales may lie as far
 * apart as that: a key's share in the softmax does not depend on its value's.  A query row with an infinity or a NaN gives NaN, and
 * no other row does.
 *
 * workspace: device, 256-byte aligned, pa_q8_workspace_bytes(); its first
 * pa_q8_workspace_zero_bytes() bytes (the same for all sizes) zero before the
 * first use, and every call that completes leaves them zero: calls of any
 * sizes that it is large enough for may use it one after another.  Calls that
 * may overlap on the GPU need workspaces of their own.  Limits: NQ <= PA_MAX_NQ, H / KV * NQ <= 1024;
 * with `selected` B * KV <= 4096; B * KV * ceil(H / KV * NQ / 8) * (capacity / 32
 * + 64) < 2^31 (PA_ERR_BAD_DIMS), capacity being max_blocks, or budget, * BLOCK.
 */
typedef struct pa_q8_opts {
    int max_blocks, num_blocks, dtype;
    int causal;
    const int32_t *selected; /* or NULL: every block */
    const int32_t *counts;
    int budget;              /* row stride of selected */
    void *workspace;
    size_t workspace_bytes;
    int *status;
} pa_q8_opts;

int pa_q8_decode(const void *q, const int8_t *k_cache, const int8_t *v_cache,
                 const float *k_scale, const float *v_scale, const int32_t *block_table,
                 const int32_t *seq_lens, void *out, float scale, int B, int H, int KV, int D,
                 int NQ, int BLOCK, const pa_q8_opts *opts, void *stream);

/* 0 for sizes that pa_q8_decode refuses (and for B == 0). */
size_t pa_q8_workspace_bytes(int B, int H, int KV, int D, int NQ);
size_t pa_q8_workspace_zero_bytes(int B, int H, int KV, int D, int NQ);

#ifdef __cplusplus
}
#endif

#endif /* PA_Q8_H */
