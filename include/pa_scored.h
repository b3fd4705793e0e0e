/*
 * pa_scored.h -- C ABI of decode attention with modified scores: capped by a
 * tanh, biased by distance, limited to a sliding window beside a prefix; and
 * of the weight that each cached key got.
 *
 * As pa_decode, with row r of sequence b at position i = seq_lens[b] + r and
 * key j at position j:
 *
 *   t = scale * q[b][h][r] . key_j
 *   t = softcap * tanh(t / softcap)                    if softcap > 0
 *   t = t - slopes[h] * |i - j|                        if slopes
 *   key j is visible to row r when j < seq_lens[b] + NQ and
 *       j < prefix[b], or
 *       (j <= i or not causal) and (|i - j| < window or window == 0)
 *   out[b][h][r] = sum_j softmax_j(t) * value_j over the visible keys
 *
 * Positions are places in the cache: behind an eviction (pa_evict.h) the kept
 * tokens stand closer together than they did in the text.
 *
 * So prefix[b] is a prefix mask: those keys are visible to every row, also
 * across the causal rule and the window (a bidirectional prompt, or the first
 * tokens kept beside a sliding window).  Every row sees its own key.  Cache
 * blocks that lie wholly between the prefix and the window of the first row
 * are not read, and keys that no row of the sequence sees have no effect
 * whatever they hold (a key that some row sees is used with weight 0 for the
 * others: its value must be finite).
 *
 * Key weights (weights != NULL): with p the softmax weights,
 *
 *   out[b][j] = decay * in[b][j] + sum_{h, r} p[b][h][r][j]   for j < seq_lens[b]
 *   out[b][j] =                    sum_{h, r} p[b][h][r][j]   for the new rows' keys
 *
 * in and out are float32 [B][max_blocks * BLOCK] and may be the same array; in
 * may be NULL (zeros); keys at max_blocks * BLOCK and beyond are dropped and
 * entries behind the last new row are left as they were.  The sums over heads
 * and rows are formed in one order, so equal calls give equal weights; a call
 * that is split otherwise (opts->partitions, another batch) has the softmax
 * denominators added in other groups, and weights that differ by their rounding
 * (a few 1e-6 of a weight).
 *
 * Layouts, ownership, streams, opts and errors as pa_decode, with these
 * differences: the batch's lengths have to fit beside two pipeline stages in
 * shared memory (any batch up to 1500; up to 4096 with few new rows), else
 * PA_ERR_UNSUPPORTED; opts->partitions must be 0 or 1 and opts->merge_kernel 0
 * (PA_ERR_UNSUPPORTED); opts->inputs_unchanged and opts->kernel are ignored.
 * slopes [H] float32 and prefix [B] int32 are device pointers or NULL (a
 * negative prefix counts as 0).  PA_ERR_BAD_DIMS: a softcap that is negative,
 * not finite, or so small or so large that |scale| / softcap is outside 2^-100
 * .. 2^100 (scale not 0) or softcap * log2(e) overflows -- a cap that is to
 * change nothing is 0 --, a negative window, a decay that is not finite, weights in and out that overlap without being one
 * array, scores whose scratch passes 2^40 bytes.  PA_ERR_NULL_POINTER: weights without out.
 * PA_ERR_WORKSPACE / PA_ERR_ALIGNMENT: scratch below
 * pa_scored_scratch_bytes() or not 256-byte aligned.  Two calls that run at
 * the same time need a workspace and a scratch each.
 */
#ifndef PA_SCORED_H
#define PA_SCORED_H

#include <stddef.h>
#include <stdint.h>

#include "pa_attention_vjp.h"
#include "pa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pa_score {
    float softcap;         /* 0: no cap */
    int window;            /* 0: no window */
    const float *slopes;   /* device [H], or NULL */
    const int32_t *prefix; /* device [B], or NULL */
} pa_score;

typedef struct pa_key_weights {
    const float *in;
    float *out;
    float decay;
    void *scratch; /* device scratch, 256-byte aligned, contents ignored */
    size_t scratch_bytes;
} pa_key_weights;

int pa_decode_scored(const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *block_table, const int32_t *seq_lens, const void *k_new,
                     const void *v_new, void *out, float scale, int H, int KV, int D, int BLOCK,
                     int NQ, int causal, const pa_score *score, const pa_key_weights *weights,
                     const pa_opts *opts, void *stream);

/* Scratch bytes of the key weights: a float32 score for every row and every
 * token that the table can hold (max_blocks * BLOCK + NQ, whatever the lengths
 * and the window: 64 sequences, 32 heads, one new row and tables of 131072
 * tokens take 1.07 GB), and the rows' softmax denominators.  0 for invalid
 * sizes. */
size_t pa_scored_scratch_bytes(int batch, int max_blocks, int BLOCK, int H, int KV, int NQ);

/*
 * The gradient of dense attention with modified scores: pa_attention_vjp
 * (pa_attention_vjp.h: arguments, layouts, opts, workspace, errors) of
 *
 *   y = softmax(score(scale * q k^T) + mask) v
 *
 * with row i and key j at positions i and j (top-left aligned, as that
 * entry's causal rule), key j visible when j < prefix[b], or j <= i (causal)
 * and |i - j| < window, and
 *
 *   ds = p * (dp - delta) * (1 - tanh^2(scale q.k / softcap))   under a cap.
 *
 * A mask of opts (mask_kind != 0) adds its bias to the modified score and
 * hides what it hides, prefix or not.  Rows that see no key get dq = 0.  The v
of a key that no row sees may hold anything; q, k, y and g must be finite.
 * 16-bit inputs with D = 128 and no mask run on the tensor cores; tiles
 * outside prefix and window are skipped.  opts->workspace holds
 * pa_attention_vjp_scored_workspace_bytes() for the current device (partial dk
 * and dv of a small call come on top of pa_attention_vjp's).  dq is accumulated by float32
 * reductions whose order varies: its last bits may differ from call to call.
 * More errors: PA_ERR_NULL_POINTER without score, PA_ERR_BAD_DIMS for a
 * softcap as above or a negative window,
 * PA_ERR_ALIGNMENT for slopes or prefix not 4-byte aligned.
 */
int pa_attention_vjp_scored(const void *q, const void *k, const void *v, const void *y,
                            const void *g, const void *mask, void *dq, void *dk, void *dv,
                            float scale, int B, int HQ, int HK, int SQ, int SK, int D,
                            const pa_score *score, const pa_vjp_opts *opts, void *stream);

size_t pa_attention_vjp_scored_workspace_bytes(int B, int HQ, int HK, int SQ, int SK, int D, int dtype,
                                               int out_dtype);

#ifdef __cplusplus
}
#endif

#endif /* PA_SCORED_H */
