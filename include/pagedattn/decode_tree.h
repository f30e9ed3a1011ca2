/*
 * libpagedattn -- decode attention for trees of drafted tokens, and keeping the
 * accepted ones. Ownership, streams, errors, layouts and tracing are as
 * pagedattn.h describes.
 */
#ifndef PAGEDATTN_DECODE_TREE_H
#define PAGEDATTN_DECODE_TREE_H

#include "../pagedattn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PA_TREE_MAX_WORDS 16    /* 64-bit mask words of a query token */
#define PA_KEEP_MAX_TOKENS 1024 /* places of a list of kept tokens */

/*
 * Decode attention of a tree of new tokens per sequence: the verification pass of
 * speculative decoding where several continuations are drafted at once
 * ("Implementation Details", Speculative Decoding -- EAGLE Proposer: draft tokens
 * proposed, then verified by the target model; pa_decode_multi is the same for
 * one continuation of a few tokens).
 *
 * q and out are [total_q, num_q_heads, head_dim] bf16, rows packed sequence after
 * sequence as in pa_prefill: sequence s owns rows [query_start_loc[s],
 * query_start_loc[s + 1]), n of them. Its nodes are the last n of its
 * L = context_lens[s] tokens in the cache, in the order of its rows (stored
 * before the call, e.g. by pa_append_kvcache with the positions of their depths).
 * Row i sees every token t < L - n, and node j (token L - n + j) where bit j % 64 of
 * tree_mask[query_start_loc[s] + i][j / 64] is set: its ancestors and itself.
 * tree_mask is [total_q, mask_words] uint64; nodes past its 64 mask_words bits are
 * seen by no row. For query head h, with K_t, V_t of KV head h / (num_q_heads /
 * num_kv_heads) gathered as in pa_decode,
 *   out = sum over the tokens seen of softmax(scale * q . K_t) V_t,
 * scores, maxima, sums and outputs held in fp32, the weights rounded to bf16 for
 * the product with V. A row that sees no token outputs zero. Any mask is taken, not
 * only a tree's; bits of nodes n and up are not read.
 *
 * What a row does not see never enters its result, whatever the cache holds there
 * (infinities and NaN of padding nodes that were not stored, of other branches).
 *
 * Rows of out outside [query_start_loc[0], query_start_loc[num_seqs]) (the
 * padding of a batch of fixed size) are not written, and nothing of them enters a
 * result. Values of query_start_loc are clamped to [0, total_q]; where one decreases,
 * results are unspecified, or not written, and stay within the buffers. With n above L,
 * tokens before the first do not exist. The call plans on the device, so a captured call follows the
 * contents of its arrays; results do not depend on timing.
 *
 * Requirements: pa_decode's for heads, blocks, pools and alignment (either layout);
 * 1 <= mask_words <= PA_TREE_MAX_WORDS; tree_mask 8-byte aligned; total_q * num_q_heads
 * below 2^31; tables of at most 2^31 - 128 tokens, and (num_seqs + total_q * g / 256) *
 * num_kv_heads * (tokens of a table / 128 + 8) below 2^31, with g the group size rounded
 * up to a power of two; a workspace of
 * pa_decode_tree_workspace_size(...) bytes, 16-byte aligned.
 */
PA_API size_t pa_decode_tree_workspace_size(int num_q_heads, int num_kv_heads, int head_dim);
PA_API pa_status_t pa_decode_tree(const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *block_tables, int max_blocks_per_seq,
                                  const int32_t *context_lens, const int32_t *query_start_loc,
                                  const uint64_t *tree_mask, int mask_words, float scale, void *out,
                                  int num_seqs, int total_q, int num_q_heads, int num_kv_heads,
                                  int head_dim, int block_size, int64_t num_blocks,
                                  pa_layout_t layout, void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * Keep the accepted tokens of every sequence's draft: with n and L as above (n from
 * query_start_loc, the last n of L = context_lens[s] tokens) and a the number of
 * leading entries of kept[s][0 .. max_kept) that are not -1, in every pool the rows of
 * token L - n + kept[s][i] become those of token L - n + i for every i < a, and
 * context_lens[s] becomes L - n + a. kept is [num_seqs, max_kept] int32; the entries
 * of a sequence ascend (a path of a tree whose nodes come after their parents): one
 * that does not, or is outside [0, n), ends the list like -1 and is recorded
 * (code 5). A sequence with n = 0 is left as it is. The caller writes the path's
 * tokens in blocks of the sequence's own (pa_fork_blocks leaves the last block so).
 *
 * With ref_counts [num_blocks] (pagedattn/blocks.h), the owned entries that the shorter
 * length no longer needs become 0 and their blocks' counts go down by one, as by
 * pa_free_blocks; with NULL the table stays as it is and the blocks are the caller's.
 * A row whose token lies in block 0 or outside the pool is skipped and recorded (5), as
 * are an entry outside the pool and a count that is already 0.
 *
 * caches, num_caches as in pagedattn/blocks.h. n above L or a negative start counts as
 * an empty draft. Requirements: pagedattn/blocks.h's; 1 <= max_kept <=
 * PA_KEEP_MAX_TOKENS; num_seqs at most 65535.
 */
PA_API pa_status_t pa_keep_tokens(void *const *caches, int num_caches, int32_t *block_tables,
                                  int max_blocks_per_seq, int32_t *context_lens,
                                  const int32_t *query_start_loc, const int32_t *kept, int max_kept,
                                  int num_seqs, int32_t *ref_counts, int num_kv_heads, int head_dim,
                                  int block_size, int64_t num_blocks, pa_layout_t layout,
                                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_DECODE_TREE_H */
