/*
 * libpagedattn -- decode attention for sequences that share a prefix.
 * Ownership, streams, errors, layouts and tracing are as pagedattn.h describes.
 */
#ifndef PAGEDATTN_DECODE_SHARED_H
#define PAGEDATTN_DECODE_SHARED_H

#include "../pagedattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Single-token decode attention (pa_decode) for a batch whose sequences come in
 * groups that share their first blocks: a system prompt or a document in front
 * of many sequences, parallel samples of one prompt, beams. The prefix of a
 * group is read and multiplied once for all its sequences ("Implementation
 * Details", PagedAttention -- the block-hash map of prefix caching lets several
 * sequences point at the same physical blocks).
 *
 * group_starts [num_groups + 1] int32, non-decreasing: group g is the sequences
 * [group_starts[g], group_starts[g + 1]). prefix_blocks [num_groups] int32: the
 * first prefix_blocks[g] table entries of all its sequences name the same
 * blocks (the call reads them through one of the group's non-empty sequences).
 * A sequence may be shorter than the prefix, or empty. Groups of one sequence
 * and prefixes of 0 blocks are plain decode. Both arrays lie on the device, so a
 * captured call follows their contents.
 *
 * What is computed together ends at the shortest non-empty sequence of a group,
 * rounded down to 16 tokens: one that is much shorter than the prefix makes all
 * the others read the rest of it by themselves. Give such a sequence a group of
 * its own. The call plans on the device, which takes a few microseconds: a batch
 * with few sequences a group and short prefixes is faster through pa_decode.
 *
 * For every sequence of a group the result is pa_decode's: the sum over the same
 * tokens t < context_lens[s], from the bf16 inputs, rounded to bf16, in another
 * order. Scores, running maxima, sums and outputs are held in fp32; as in
 * pa_decode the softmax weights are rounded to bf16 for the product with V. The
 * sum of the weights is of the rounded ones where a sequence reads its tokens by
 * itself or with a few others, and of the exact ones where a prefix is computed
 * for many. Sequences outside all groups (before group_starts[0], or from
 * group_starts[num_groups] on: the padding of a batch of fixed size) are not
 * written, and nothing of them enters a result.
 *
 * Values of group_starts are clamped to [0, num_seqs] and prefixes to the
 * table's width; a group_starts that decreases gives unspecified results within
 * the buffers. Requirements: pa_decode's; num_groups at most 4096, num_seqs and
 * num_kv_heads at most 65535; tables of at most 2^31 - 128 tokens
 * (max_blocks_per_seq * block_size); pools in either layout; a workspace of
 * pa_decode_shared_workspace_size(num_seqs, num_groups, ...) bytes, 16-byte
 * aligned. Results do not depend on timing.
 */
PA_API size_t pa_decode_shared_workspace_size(int num_seqs, int num_groups, int num_q_heads,
                                              int num_kv_heads, int head_dim);
PA_API pa_status_t pa_decode_shared(const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *block_tables, int max_blocks_per_seq,
                                    const int32_t *context_lens, const int32_t *group_starts,
                                    const int32_t *prefix_blocks, int num_groups, float scale,
                                    void *out, int num_seqs, int num_q_heads, int num_kv_heads,
                                    int head_dim, int block_size, int64_t num_blocks,
                                    pa_layout_t layout, void *workspace, size_t workspace_bytes,
                                    void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_DECODE_SHARED_H */
