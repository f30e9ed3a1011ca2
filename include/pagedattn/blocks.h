/*
 * libpagedattn -- operations on the blocks of the paged KV cache: copying,
 * forking and freeing sequences' blocks, compacting the pools. Ownership,
 * streams, errors, layouts and tracing are as pagedattn.h describes.
 */
#ifndef PAGEDATTN_BLOCKS_H
#define PAGEDATTN_BLOCKS_H

#include "../pagedattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Operations on the blocks of the pools.
 *
 * A table row owns its first ceil(context_lens[row] / block_size) entries (a
 * length is clamped to [0, max_blocks_per_seq * block_size]), and
 * ref_counts [num_blocks] int32 holds for every block the number of owned
 * entries that name it: blocks with count 0 are free. Block 0 is the null
 * block: it may stand in a table, but is never handed out, moved or counted.
 * Tables, lengths and counts are the caller's device memory, kept from call to
 * call; a caller that hands out blocks itself sets their counts.
 *
 * caches is a host array of num_caches device pointers to the pools that are
 * indexed by the same block ids, normally the K and the V pool of every layer,
 * all of the shape the other arguments give; it is read before the call
 * returns. A pool may be listed once. With num_caches == 0 fork and compact
 * change tables, lengths and counts only.
 *
 * Requirements of all four: head_dim == 128; block_size a power of two in
 * [16, 256]; num_blocks in [1, 2^31); num_kv_heads at most 65535; pools
 * 16-byte aligned. Ids that are read on the device are never trusted for
 * addressing: what is out of range is skipped and recorded for
 * pa_take_device_error. Calls that share tables, counts or pools are ordered
 * by the caller, normally by the stream.
 */

/*
 * Copy blocks: for every i < num_pairs, block block_pairs[i][1] of every pool
 * becomes a copy of block block_pairs[i][0], bit by bit. block_pairs is
 * [num_pairs, 2] int32 on the device, 8-byte aligned; a pair with an id of -1
 * is skipped. A block that one pair writes must not stand in another pair
 * (what is left there is unspecified). Tables and counts are not touched.
 */
PA_API pa_status_t pa_copy_blocks(void *const *caches, int num_caches, const int32_t *block_pairs,
                                  int64_t num_pairs, int num_kv_heads, int head_dim,
                                  int block_size, int64_t num_blocks, void *stream);

/*
 * Bytes of workspace pa_fork_blocks and pa_compact_blocks need for tables of
 * num_rows rows over num_blocks blocks; 0 for sizes they do not take. The
 * workspace needs no initialisation and holds nothing after the call.
 */
PA_API size_t pa_blocks_workspace_size(int num_rows, int64_t num_blocks);

/*
 * Fork sequences: for every i < num_forks, row children[i] becomes a second
 * sequence with the tokens of row parents[i] (parallel samples of a prompt,
 * beams). With L the parent's length as it was before the call:
 *   - the child's length becomes L and its owned entries the parent's;
 *   - every full block among them is shared, its count one higher;
 *   - a partly filled last block is not shared: the child gets a free block
 *     with count 1 and, in every pool, a copy of the L % block_size used rows.
 *     The forks that need a block take the lowest free ids, in the order of i.
 * So a sequence's partly filled block is its own alone, and its next token can
 * be stored without a copy. Entries of the child past its owned ones and the
 * unused rows of its new block are left as they were.
 *
 * The child row must be empty (length 0 or less), and is given to the first
 * fork that lists it; a fork whose child is not empty or was listed before, or
 * that finds no free block, changes nothing and is recorded (code 6). A parent
 * or child of -1 is skipped. Owned entries that are 0, outside the pool or name a
 * block with count 0 are passed on as they are, the last one too: no block is
 * taken and no row copied for it. A block with count 0 is free whatever names
 * it: the same call may hand it to a fork as its new block. Its count is then 1
 * for that fork and 1 more for each entry passed on, and a full block's entry
 * that names it is not recorded.
 *
 * num_forks is at most num_rows. Workspace: pa_blocks_workspace_size(num_rows,
 * num_blocks) bytes, 16-byte aligned. `layout` is the pools'.
 */
PA_API pa_status_t pa_fork_blocks(void *const *caches, int num_caches, int32_t *block_tables,
                                  int max_blocks_per_seq, int32_t *context_lens, int num_rows,
                                  int32_t *ref_counts, const int32_t *parents,
                                  const int32_t *children, int num_forks, int num_kv_heads,
                                  int head_dim, int block_size, int64_t num_blocks,
                                  pa_layout_t layout, void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * Free sequences: every listed row gives up its owned entries. Each named
 * block's count goes down by one, the entries become 0 and the length 0. A row
 * of -1 is skipped; a row listed twice is freed once; a count that is already
 * 0 stays 0 and is recorded. The pools are not touched.
 */
PA_API pa_status_t pa_free_blocks(int32_t *block_tables, int max_blocks_per_seq,
                                  int32_t *context_lens, int num_rows, int32_t *ref_counts,
                                  const int32_t *rows, int num_freed, int block_size,
                                  int64_t num_blocks, void *stream);

/*
 * Compact the pools: with n live blocks (count above 0; the null block is none
 * of them) the live ids become 1 .. n. The k-th lowest live id above n moves to
 * the k-th lowest free id up to n, in every pool; no other block moves. Counts
 * and the owned entries of all num_rows rows follow; *num_live becomes n and
 * remap [num_blocks] the new id of every live block (its own if it stayed) and
 * 0 for the others, so that a caller can carry over ids it keeps elsewhere. An
 * owned entry that is outside the pool or names a block with count 0 is left
 * as it is and recorded. The contents of the blocks that became free are
 * unspecified.
 *
 * remap and num_live are device memory. Workspace as for pa_fork_blocks.
 */
PA_API pa_status_t pa_compact_blocks(void *const *caches, int num_caches, int32_t *block_tables,
                                     int max_blocks_per_seq, const int32_t *context_lens,
                                     int num_rows, int32_t *ref_counts, int32_t *remap,
                                     int32_t *num_live, int num_kv_heads, int head_dim,
                                     int block_size, int64_t num_blocks, void *workspace,
                                     size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_BLOCKS_H */
