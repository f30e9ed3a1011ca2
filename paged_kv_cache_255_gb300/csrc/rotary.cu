// Rotary positions: the rotation of query and key heads, with the norm of each
// head's row before it in the same pass, and the append of a step's keys and
// values to the paged pools with both on the way ("A vLLM engine small enough to
// read in one sitting", paged KV cache management: the projections of a step's
// tokens are stored before attention reads them back).
//
//   y = x w / sqrt(mean(x^2) + eps);  (a, b) -> A (a cos px - b sin px, b cos px + a sin px)
//
// The angle: pair i turns F_i 2^-64 of a circle per token, F_i a 64-bit whole
// number, so the low 64 bits of p F_i are the angle modulo one turn for any 32-bit
// position p, with an error of p 2^-64 turns (the frequency in fp32 would be off by
// a tenth of a radian at p = 2^20). Its upper 32 bits as a signed fraction go to
// sincospif, whose argument then needs no reduction.
//
// One row of 256 bytes is 8 lanes' work: a lane holds 8 pairs, which are two
// 16-byte chunks (neighbours when interleaved, rot_dim / 2 dims apart otherwise), so
// a pair never leaves its lane; a warp works on four rows at a time. The 64 sines
// and cosines of a token are computed once per warp, two pairs a lane, handed round
// by shuffles, and used for all heads the warp takes.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.h"
#include "rotary.h"

namespace pa {

__device__ int g_rotary_error;       // first device-side error of an append

namespace {

constexpr int kWarps = 4;
constexpr int kChunks = kHeadDim / 8;       // 16-byte chunks of a row
constexpr int kBatch = 2;                   // quads of heads whose loads are in flight together

__device__ __forceinline__ void unpack(const uint4 &w, float (&f)[8]) {
    f[0] = bf16_lo(w.x);
    f[1] = bf16_hi(w.x);
    f[2] = bf16_lo(w.y);
    f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z);
    f[5] = bf16_hi(w.z);
    f[6] = bf16_lo(w.w);
    f[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

enum Kind { kQuery, kKey, kValue };

template <bool APPEND, bool INTERLEAVED>
__global__ void __launch_bounds__(kWarps * 32)
rotate_kernel(const __grid_constant__ RotateArgs a) {
    __shared__ uint64_t s_turns[kRotaryPairs];
    const int lane = threadIdx.x & 31, sub = lane & 7;
    for (int i = threadIdx.x; i < kRotaryPairs; i += kWarps * 32) s_turns[i] = a.turns[i];
    // this lane's chunks of a row, and whether its pairs are rotated
    const bool rotated = sub * 8 < a.pairs;
    const bool apart = !INTERLEAVED && rotated;
    const int c0 = apart ? sub : 2 * sub, c1 = apart ? sub + a.pairs / 8 : 2 * sub + 1;
    // programmatic dependent of whatever precedes the call
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    uint4 qw[2] = {}, kw[2] = {};
    if (a.q_weight) {
        qw[0] = __ldg(a.q_weight + c0);
        qw[1] = __ldg(a.q_weight + c1);
    }
    if (a.k_weight) {
        kw[0] = __ldg(a.k_weight + c0);
        kw[1] = __ldg(a.k_weight + c1);
    }
    __syncthreads();
    const int hq = a.num_q_heads, hk = a.num_kv_heads, rows = hq + hk + (APPEND ? hk : 0);
    const int64_t items = a.num_tokens * a.slices;
    const int64_t stride = (int64_t)gridDim.x * kWarps;
    for (int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); item < items; item += stride) {
        const int64_t t = item / a.slices;
        const int first = (int)(item - t * a.slices) * a.quads * 4;
        const int last = first + a.quads * 4 < rows ? first + a.quads * 4 : rows;
        int64_t slot = 0;
        bool stored = false;
        if (APPEND) {
            slot = __ldg(a.slots + t);
            stored = slot >= 0 && slot < a.num_slots;
            if (!stored && slot != -1 && lane == 0) atomicCAS(&g_rotary_error, 0, kErrBadSlot);
        }
        const int p = a.positions ? __ldg(a.positions + t) : 0;
        float cs[8], sn[8];
        bool have = false;
        for (int h0 = first; h0 < last; h0 += 4 * kBatch) {
            uint4 x[kBatch][2];
            uint4 *out[kBatch];
            Kind kind[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int h = h0 + 4 * b + (lane >> 3);
                const uint4 *src = nullptr;
                out[b] = nullptr;
                kind[b] = h < hq ? kQuery : (h < hq + hk ? kKey : kValue);
                if (h < last) {
                    const HeadRows &r = kind[b] == kQuery ? a.q : (kind[b] == kKey ? a.k : a.v);
                    const int head = kind[b] == kQuery ? h : (kind[b] == kKey ? h - hq : h - hq - hk);
                    src = r.p + t * r.token + head * r.head;
                    if (kind[b] == kQuery) {
                        out[b] = a.q_out.p + t * a.q_out.token + head * a.q_out.head;
                    } else if (!APPEND) {
                        out[b] = a.k_out.p + t * a.k_out.token + head * a.k_out.head;
                    } else if (stored) {
                        const int lb = a.block_size_log2;
                        const int64_t row = a.head_major
                            ? (((slot >> lb) * hk + head) << lb) + (slot & ((1 << lb) - 1))
                            : slot * hk + head;
                        out[b] = (kind[b] == kKey ? a.k_cache : a.v_cache) + row * kChunks;
                    }
                }
                if (out[b]) {
                    x[b][0] = src[c0];
                    x[b][1] = src[c1];
                } else {
                    x[b][0] = x[b][1] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            if (a.positions && !have) {
                // pairs 2 lane and 2 lane + 1, then each lane the 8 of its own
                have = true;
                float c2[2], s2[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint64_t turn = (uint64_t)(int64_t)p * s_turns[2 * lane + k];
                    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s2[k], &c2[k]);
                    s2[k] *= a.amplitude;
                    c2[k] *= a.amplitude;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    cs[j] = __shfl_sync(0xffffffffu, c2[j & 1], 4 * sub + (j >> 1));
                    sn[j] = __shfl_sync(0xffffffffu, s2[j & 1], 4 * sub + (j >> 1));
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const bool key = kind[b] == kKey;
                const bool norm = kind[b] != kValue && (key ? a.k_weight : a.q_weight) != nullptr;
                const bool turn = kind[b] != kValue && rotated;
                float f[2][8];
                unpack(x[b][0], f[0]);
                unpack(x[b][1], f[1]);
                float sq = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sq = fmaf(f[0][i], f[0][i], fmaf(f[1][i], f[1][i], sq));
#pragma unroll
                for (int m = 1; m < 8; m <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
                if (norm) {
                    const float inv = rsqrtf(fmaf(sq, 1.f / kHeadDim, a.eps));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float w[8];
                        unpack(key ? kw[k] : qw[k], w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[k][i] *= inv * w[i];
                    }
                }
                if (turn) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float &u = INTERLEAVED ? f[j >> 2][2 * (j & 3)] : f[0][j];
                        float &v = INTERLEAVED ? f[j >> 2][2 * (j & 3) + 1] : f[1][j];
                        const float n = u * cs[j] - v * sn[j];
                        v = v * cs[j] + u * sn[j];
                        u = n;
                    }
                }
                if (out[b]) {
                    // neither normed nor rotated: the bits as they are
                    out[b][c0] = norm || turn ? pack(f[0]) : x[b][0];
                    out[b][c1] = norm || turn ? pack(f[1]) : x[b][1];
                }
            }
        }
    }
}

template <bool APPEND, bool INTERLEAVED>
cudaError_t launch(const RotateArgs &a, unsigned grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rotate_kernel<APPEND, INTERLEAVED>, a);
}

}  // namespace

void rotary_fill(pa_rotary_t *r, int rot_dim, int interleaved, const double *radians, double amplitude) {
    std::memset(r, 0, sizeof(*r));
    r->rot_dim = rot_dim;
    r->interleaved = interleaved ? 1 : 0;
    r->amplitude = (float)amplitude;
    for (int i = 0; i < rot_dim / 2; ++i) {
        double turns = radians[i] / (2 * 3.14159265358979323846);
        turns -= std::floor(turns);             // of one turn; 1.0 where it rounds up to a whole one
        r->turns[i] = turns < 1.0 ? (uint64_t)std::ldexp(turns, 64) : 0;
    }
}

void rotary_scaled(double *radians, int rot_dim, double base, pa_rotary_scaling_t scaling, double factor,
                   double original_context, double low, double high) {
    const double circle = 2 * 3.14159265358979323846;
    if (scaling == PA_ROTARY_NTK) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    // index of the pair that turns n times in the original context
    auto index = [&](double n) {
        return rot_dim * std::log(original_context / (n * circle)) / (2 * std::log(base));
    };
    double first = 0, last = 0;
    if (scaling == PA_ROTARY_YARN) {
        first = std::max(std::floor(index(high)), 0.0);
        last = std::min(std::ceil(index(low)), rot_dim - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double theta = std::pow(base, -2.0 * i / rot_dim);
        double keep = 1;                        // share of theta; the rest is of theta / factor
        if (scaling == PA_ROTARY_LINEAR) keep = 0;
        if (scaling == PA_ROTARY_YARN) keep = 1 - (i - first) / std::max(last - first, 1e-3);
        if (scaling == PA_ROTARY_BANDED) keep = (original_context * theta / circle - low) / (high - low);
        keep = std::min(std::max(keep, 0.0), 1.0);
        const double slow = scaling == PA_ROTARY_PLAIN || scaling == PA_ROTARY_NTK ? theta : theta / factor;
        radians[i] = slow * (1 - keep) + theta * keep;
    }
}

cudaError_t take_rotary_error(cudaStream_t stream, int *code) {
    return take_device_word(g_rotary_error, stream, code);
}

cudaError_t launch_rotate(RotateArgs a, bool append, bool interleaved, int sm_count, cudaStream_t stream) {
    const int rows = a.num_q_heads + a.num_kv_heads * (append ? 2 : 1);
    const int all = (rows + 3) / 4;             // quads of a token
    // A warp takes as many of a token's quads as leave the GPU full of warps: the
    // sines are then computed once for all of them.
    const int64_t full = (int64_t)sm_count * 32;
    int64_t quads = a.num_tokens * all / full;
    a.quads = (int)(quads < 1 ? 1 : (quads > all ? all : quads));
    a.slices = (all + a.quads - 1) / a.quads;
    int64_t grid = (a.num_tokens * a.slices + kWarps - 1) / kWarps;
    const int64_t most = (int64_t)sm_count * 16;
    if (grid > most) grid = most;
    if (append)
        return interleaved ? launch<true, true>(a, (unsigned)grid, stream)
                           : launch<true, false>(a, (unsigned)grid, stream);
    return interleaved ? launch<false, true>(a, (unsigned)grid, stream)
                       : launch<false, false>(a, (unsigned)grid, stream);
}

}  // namespace pa
