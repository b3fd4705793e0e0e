/*
 * pa_rotary.h -- C ABI of the rotary position embedding: queries and new keys
 * turned by their positions, the gradient of that, and the same fused with the
 * store of the step's new rows into the paged cache.
 *
 * For row n of sequence b, pair i of the first `rot` columns of every head:
 *
 *   phase = positions[b][n] * table[i]  mod 2^64      (2^64 = one turn)
 *   theta = 2 pi phase / 2^64
 *   (u, v) -> factor * (u cos(theta) - v sin(theta), u sin(theta) + v cos(theta))
 *
 * where the pair (u, v) is columns (i, i + rot / 2), or (2 i, 2 i + 1) with
 * opts->interleaved.  Columns rot .. D-1 are copied.  opts->inverse turns by
 * -theta: with the same factor, that is the gradient (the transpose) of the
 * forward call.  table[i] is the angle per position in turns, as a 64-bit
 * fixed-point fraction: the product with a 32-bit position wraps at whole
 * turns, so far positions lose nothing (the angle is exact to 2^-32 turns).
 * Negative positions turn backwards.
 *
 * Layouts (elements; device memory):
 *   q       [B][H][N][D] with strides opts->q_strides = {batch, head, row}
 *   k, v    [B][KV][N][D] with opts->k_strides, opts->v_strides; columns are
 *           contiguous, every stride a multiple of 16 bytes
 *   q_out   [B][H][N][D], k_out [B][KV][N][D] contiguous
 *   positions [B][N] int32, table [rot / 2] uint64
 * H or KV may be 0 (then q / k and their outputs may be NULL).  An output may
 * not overlap an input.
 *
 * Cache store (opts->slot_mapping != NULL): v has the layout of k;
 * slot_mapping [B][N] int32 as in pa_cache_append (slot = physical block *
 * BLOCK + offset, -1 stores nothing, any other slot outside the pool is
 * skipped and reported as PA_STATUS_BAD_SLOT; of several rows of one sequence
 * bound for one slot the last is stored): the rotated key goes to k_cache, the
 * value as it is to v_cache, each [num_blocks][BLOCK][KV][D].  k_out may then
 * be NULL.
 *
 * Every call is asynchronous on `stream`; the library keeps nothing.  Returns
 * PA_OK or a PA_ERR_* code of pa_decode.h before anything is launched:
 *   PA_ERR_NULL_POINTER  a needed pointer is NULL
 *   PA_ERR_BAD_DIMS      a size < 0, H + KV < 1, D < 1, rot odd or outside
 *                        [2, D], a factor that is not finite, an output that
 *                        overlaps an input, 2^31 rows (B * N) or more
 *   PA_ERR_UNSUPPORTED   a dtype outside PA_F32, PA_F16, PA_BF16; rows that
 *                        are not a multiple of 16 bytes; D > 1024;
 *                        N > PA_MAX_PREFILL with a cache store
 *   PA_ERR_ALIGNMENT     a tensor not 16-byte aligned, a stride not a
 *                        multiple of 16 bytes or negative
 * Arithmetic: float32 (cos and sin to about one unit in the last place of the
 * exact angle), one rounding to the dtype.
 */
#ifndef PA_ROTARY_H
#define PA_ROTARY_H

#include <stddef.h>
#include <stdint.h>

#include "pa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pa_rotary_opts {
    int dtype;       /* PA_F32, PA_F16, PA_BF16: every tensor of rows */
    int interleaved; /* 1: pairs (2 i, 2 i + 1); 0: pairs (i, i + rot / 2) */
    int inverse;     /* 1: turn by -theta (the gradient) */
    float factor;    /* multiplies the rotated columns */
    long long q_strides[3], k_strides[3], v_strides[3]; /* elements: batch, head, row */
    /* cache store: all unused when slot_mapping is NULL */
    const int32_t *slot_mapping; /* [B][N] */
    const void *v;
    void *k_cache;
    void *v_cache;
    int BLOCK, num_blocks;
    int *status; /* device int32 for PA_STATUS_BAD_SLOT, or NULL */
} pa_rotary_opts;

int pa_rotary(const void *q, const void *k, const int32_t *positions, const uint64_t *table,
              void *q_out, void *k_out, int B, int H, int KV, int N, int D, int rot,
              const pa_rotary_opts *opts, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_ROTARY_H */
