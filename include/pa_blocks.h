/*
 * pa_blocks.h -- C ABI of the block manager of a paged cache: the block tables
 * of a serving step and the slots of its new rows, made on the device from the
 * sequences' lengths.
 *
 * For every sequence b, with n = seq_lens[b] tokens in the cache, keep[b] of
 * them to stay (keep NULL: n; 0 for a sequence that is done) and add[b] new
 * ones (add NULL: N):
 *
 *   have = ceil(n / BLOCK)                blocks that it has, block_table[b][0 .. have-1]
 *   need = ceil((keep + add) / BLOCK)     blocks that it needs
 *   need < have: block_table[b][need .. have-1] go back to the free blocks
 *   need > have: block_table[b][have .. need-1] are taken from the free blocks
 *
 * free_blocks[0 .. free_count-1] is a stack.  The blocks given back by all
 * sequences are put on top of it in the order of the sequences (and of their
 * places in the table); then the blocks taken come off its top in the order of
 * the sequences that need them.  A sequence whose blocks, added to those taken
 * by the sequences before it, exceed what there is, is refused, and with it
 * every later one that needs a block; one that would need more than max_blocks
 * is refused by itself.  A refused sequence is left as it was, with n tokens.
 *
 *   new_lens[b]       keep + add, or n when refused
 *   new_free_count    free blocks left on the stack
 *   slots[b][j]       block_table[b][t / BLOCK] * BLOCK + t % BLOCK of token
 *                     t = keep + j for j < add, -1 behind them, when refused
 *                     and for a block outside the pool: the slot_mapping of
 *                     pa_rotary and pa_cache_append
 *   positions[b][j]   t, or starts[b] + j with starts (the place in the text,
 *                     after an eviction), for the same rows; -1 for the others
 *   kept[b]           tokens before the new rows: keep, or n when refused
 *   granted[b]        new rows that have their blocks: add, or 0 when refused
 *                     (kept + granted = new_lens)
 *
 * A store that takes lengths and counts instead of slots (pa_q8_append) is given
 * kept and granted, never keep and add: those of a refused sequence, or of one
 * whose values were clamped, name rows that are not its own (the table's entries
 * behind its blocks may be of blocks that others have by now).
 *
 * block_table and free_blocks are changed in place: the tables' entries behind
 * need stay as they were, and so do the stack's behind new_free_count but for
 * blocks that were given back.  seq_lens, free_count and the other inputs are only read:
 * a loop goes on with new_lens and new_free_count.  The call can be repeated
 * with the same inputs and gives the same result.  Blocks that two sequences
 * share must not be given back.
 *
 * Layouts (row-major, device memory, int32): block_table [B][max_blocks];
 * seq_lens, keep, add, starts, new_lens, kept, granted [B]; free_blocks [num_blocks];
 * free_count, new_free_count [1]; slots, positions [B][N].
 *
 * Conditions that only the device sees are OR-ed into *opts->status:
 *   PA_STATUS_NO_BLOCKS   a sequence was refused for want of blocks
 *   PA_STATUS_BAD_LENGTH  a length, keep, add or free_count outside its range
 *                         ([0, max_blocks * BLOCK], [0, n], [0, N],
 *                         [0, num_blocks]; clamped), a sequence that would
 *                         outgrow its table row, more blocks given back than
 *                         the stack holds (the rest are dropped)
 *   PA_STATUS_BAD_BLOCK   a block outside the pool among those taken
 *
 * Asynchronous on `stream`; the library keeps nothing and needs no workspace.
 * Returns PA_OK or, before anything is launched, a PA_ERR_* code of
 * pa_decode.h:
 *   PA_ERR_NULL_POINTER  a needed pointer is NULL (slots when N > 0)
 *   PA_ERR_BAD_DIMS      B < 0, N < 0, another size < 1, max_blocks * BLOCK >=
 *                        2^30, num_blocks * BLOCK >= 2^31, B * max_blocks >=
 *                        2^31, B * N >= 2^31, overlapping outputs
 *   PA_ERR_UNSUPPORTED   B > 4096, N > PA_MAX_PREFILL
 *   PA_ERR_ALIGNMENT     a tensor not 4-byte aligned
 */
#ifndef PA_BLOCKS_H
#define PA_BLOCKS_H

#include <stddef.h>
#include <stdint.h>

#include "pa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pa_blocks_opts {
    int max_blocks;         /* row stride of block_table */
    int num_blocks;         /* physical blocks of the pool, entries of free_blocks */
    const int32_t *add;     /* [B], or NULL: N */
    const int32_t *keep;    /* [B], or NULL: seq_lens */
    const int32_t *starts;  /* [B], or NULL: positions count the cache */
    int32_t *positions;     /* [B][N], or NULL */
    int *status;            /* device int32 for PA_STATUS_* bits, or NULL */
    int32_t *kept;          /* [B], or NULL */
    int32_t *granted;       /* [B], or NULL */
} pa_blocks_opts;

int pa_plan_blocks(int32_t *block_table, const int32_t *seq_lens, int32_t *free_blocks,
                   const int32_t *free_count, int32_t *new_lens, int32_t *new_free_count,
                   int32_t *slots, int B, int N, int BLOCK, const pa_blocks_opts *opts,
                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_BLOCKS_H */
