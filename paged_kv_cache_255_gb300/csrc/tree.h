// Decode over trees of drafted tokens, and keeping the accepted ones (tree.cu,
// keep.cu), behind the C ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace pa {

// One launch (pointers are device memory).
struct TreeArgs {
    const void *q;                  // bf16 [total_q, Hq, 128], rows packed per sequence
    const void *k_cache, *v_cache;
    const int32_t *block_tables;    // [S, max_blocks_per_seq]
    const int32_t *context_lens;    // [S], counting each sequence's nodes
    const int32_t *starts;          // [S + 1]
    const uint32_t *mask;           // [total_q, mask_words] bit j: node j is seen
    void *out;                      // bf16 [total_q, Hq, 128]
    int mask_words;                 // 32-bit words of a mask row
    int num_seqs;
    int total_q;
    int num_q_heads;
    int num_kv_heads;
    int group;
    int block_size_log2;
    int max_blocks_per_seq;
    int head_major;
    int box_tokens;                 // tokens of a TMA box: min(block size, 128)
    int fault_hold_v;               // test hook, normally 0: see set_prefill_fault
    int64_t num_blocks;
    float scale_log2;
    int workers;                    // CTAs the work is shared among
    // in the workspace
    int4 *tasks;                    // [workers] the unit that a share leaves unfinished: first query row (-1: none), KV
                                    // head, query rows, parts and (from bit 8) the workers between them
    float4 *part_o;                 // [2 workers][32][256] parts of units that several workers share
    float2 *part_ml;                // [2 workers][256] (running max in log2 units, sum)
};

// A task packs counts of workers into bytes, and the merge has a thread for each worker.
constexpr int kTreeMaxWorkers = 255;

size_t tree_workspace_bytes(int workers);
void tree_carve_workspace(TreeArgs &a, void *workspace);
cudaError_t launch_decode_tree(const TreeArgs &a, int group_pad, cudaStream_t stream);
cudaError_t take_tree_error(cudaStream_t stream, int *code);

struct KeepArgs {
    int32_t *block_tables;          // [num_seqs, max_blocks]
    int32_t *context_lens;          // [num_seqs]
    const int32_t *starts;          // [num_seqs + 1]
    const int32_t *kept;            // [num_seqs, max_kept]
    int32_t *ref_counts;            // [num_blocks] or nullptr
    int max_blocks;
    int max_kept;
    int num_seqs;
    int block_size_log2;
    int num_kv_heads;
    int head_major;
    int64_t num_blocks;
};

cudaError_t launch_keep_tokens(void *const *caches, int num_caches, const KeepArgs &a, int sm_count,
                               cudaStream_t stream);
cudaError_t take_keep_error(cudaStream_t stream, int *code);

}  // namespace pa
