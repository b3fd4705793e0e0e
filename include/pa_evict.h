/*
 * pa_evict.h -- C ABI of the cache eviction by accumulated attention weight.
 *
 * For every sequence b with n = seq_lens[b] cached tokens and a budget:
 *
 *   n <= budget: every token is kept.
 *   n >  budget: kept are the first keep_first tokens, the last keep_last, and
 *     of those between the budget - keep_first - keep_last with the largest
 *     weights[b][j] (equal weights: the lowest j first; a NaN weight counts
 *     as lower than any other; -0 equals 0).
 *   kept[b][0 .. m-1]  the kept tokens' indices in ascending order, m = min(n, budget)
 *   new_lens[b]        m
 *   weights_out[b][r]  weights[b][kept[b][r]]
 *   token r of the shortened sequence gets the K and V rows of token
 *   kept[b][r], as they are (keys keep the positions they were rotated by).
 *
 * The shortened sequence counts its tokens from 0 again: the distances of
 * pa_decode_scored (slopes, window) and its prefix are then between places in
 * the cache, r, no longer between the tokens' places in the text, kept[b][r].
 * keep_first at least as large as the prefix leaves the prefix as it was, and
 * keep_last at least as large as the window (or as the reach of the slopes)
 * leaves the distances inside it exact; older kept tokens come nearer.
 *
 * kept[b][m .. budget-1] is set to -1, weights_out[b][m .. width-1] to 0.
 *
 * The rows move inside the sequence's own blocks (dst_table NULL: token r goes
 * to the slot that block_table gives token r; slots of tokens m .. n-1 keep
 * what they held), or into the blocks of dst_table (every kept row is copied,
 * the source blocks are left as they were).  A block that several sequences
 * share must not be moved in place; dst_table serves that.  In either case no
 * two tokens' destination slots may coincide, and no block of dst_table may
 * be a block of block_table.
 *
 * Layouts (row-major, device memory):
 *   k_cache, v_cache [num_blocks][BLOCK][KV][D] of dtype, 16-byte aligned
 *   block_table [B][max_blocks], dst_table [B][dst_max_blocks] int32
 *   seq_lens, new_lens [B] int32; kept [B][budget] int32
 *   weights, weights_out [B][max_blocks * BLOCK] float32 (the accumulated
 *   weights that pa_decode_scored keeps)
 * seq_lens, weights and the tables are only read; the outputs may not overlap
 * them.  A length outside [0, max_blocks * BLOCK] is clamped and reported as
 * PA_STATUS_BAD_LENGTH; a row whose source or destination block is outside the
 * pool is not moved and reported as PA_STATUS_BAD_BLOCK.
 *
 * Asynchronous on `stream`; the library keeps nothing and needs no workspace.
 * Returns PA_OK or, before anything is launched, a PA_ERR_* code of
 * pa_decode.h:
 *   PA_ERR_NULL_POINTER  a needed pointer is NULL
 *   PA_ERR_BAD_DIMS      a size < 1 (B < 0), keep_first or keep_last < 0,
 *                        keep_first + keep_last > budget, max_blocks * BLOCK
 *                        >= 2^30, num_blocks * BLOCK >= 2^31, budget >= 2^30,
 *                        a dst_table that is block_table itself,
 *                        a dst_table too short for min(budget, max_blocks *
 *                        BLOCK) tokens, overlapping outputs
 *   PA_ERR_UNSUPPORTED   a dtype outside PA_F32, PA_F16, PA_BF16; a token row
 *                        (KV * D elements) that is not a multiple of 16 bytes
 *                        or above 64 KB; B > 4096
 *   PA_ERR_ALIGNMENT     a cache not 16-byte aligned, another tensor not
 *                        4-byte aligned
 */
#ifndef PA_EVICT_H
#define PA_EVICT_H

#include <stddef.h>
#include <stdint.h>

#include "pa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pa_evict_opts {
    int max_blocks;     /* row stride of block_table */
    int num_blocks;     /* physical blocks in each cache */
    int dtype;          /* PA_F32, PA_F16, PA_BF16 */
    int budget;         /* tokens a sequence keeps at most */
    int keep_first;     /* kept whatever they weigh */
    int keep_last;
    const int32_t *dst_table; /* NULL: in place */
    int dst_max_blocks;       /* row stride of dst_table */
    int *status;              /* device int32 for PA_STATUS_* bits, or NULL */
} pa_evict_opts;

int pa_cache_evict(void *k_cache, void *v_cache, const int32_t *block_table,
                   const int32_t *seq_lens, const float *weights, int32_t *new_lens, int32_t *kept,
                   float *weights_out, int B, int KV, int D, int BLOCK, const pa_evict_opts *opts,
                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_EVICT_H */
