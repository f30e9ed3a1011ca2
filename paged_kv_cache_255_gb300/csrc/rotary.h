// Rotation of heads (rotary.cu) behind the C ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/pagedattn/rotary.h"

namespace pa {

constexpr int kRotaryPairs = PA_ROTARY_MAX_PAIRS;

// Rows of one tensor; strides in 16-byte chunks.
struct HeadRows {
    const uint4 *p;
    int64_t token, head;
};
struct HeadRowsOut {
    uint4 *p;
    int64_t token, head;
};

// One launch over the heads of q, then k, then (append) v of every token.
// Pointers are device memory.
struct RotateArgs {
    HeadRows q, k, v;
    HeadRowsOut q_out, k_out;       // k_out: rotate only
    uint4 *k_cache, *v_cache;       // append only
    const int64_t *slots;           // append only: [num_tokens]
    int64_t num_slots;
    int block_size_log2;
    int head_major;
    const int32_t *positions;       // nullptr: nothing is rotated
    const uint4 *q_weight, *k_weight;   // nullptr: no norm
    int64_t num_tokens;
    int num_q_heads, num_kv_heads;
    int pairs;                      // rotated pairs of a head: rot_dim / 2
    int quads;                      // groups of four heads a warp takes of a token
    int slices;                     // warps a token's heads are shared among
    float amplitude, eps;
    uint64_t turns[kRotaryPairs];   // turns per token in units of 2^-64
};

// Frequencies in radians per token -> turns; host only.
void rotary_fill(pa_rotary_t *r, int rot_dim, int interleaved, const double *radians, double amplitude);
// The frequencies of a scaling whose arguments have been checked.
void rotary_scaled(double *radians, int rot_dim, double base, pa_rotary_scaling_t scaling, double factor,
                   double original_context, double low, double high);

cudaError_t launch_rotate(RotateArgs a, bool append, bool interleaved, int sm_count, cudaStream_t stream);
cudaError_t take_rotary_error(cudaStream_t stream, int *code);

}  // namespace pa
