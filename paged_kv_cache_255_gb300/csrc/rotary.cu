// Rotary positions: the rotation of query and key heads, with the norm of each
// head's row before it in the same pass, and the append of a step's keys and
// values to the paged pools with both on the way ("A vLLM engine small enough to
// read in one sitting", paged KV cache management: the projections of a step's
// tokens are stored before attention reads them back).
//
//   y = x w / sqrt(mean(x^2) + eps);  (a, b) -> A (a cos px - b sin px, b cos px + a sin px)
//
// The angle: pair i turns F_i 2^-64 of a circle per token, F_i a 64-bit whole number that
// is its frequency (a double) to half a unit, so the low 64 bits of p F_i are the angle
// modulo one turn for any 32-bit position p to |p| 2^-65 turns (the frequency in fp32
// would be off by a tenth of a radian at p = 2^20). The upper 32 bits as a signed fraction,
// rounded to fp32 (2^-26 of a turn at most), go to sincospif, whose argument then needs no
// reduction.
//
// One row of 256 bytes is 8 lanes' work: a lane holds 8 pairs, which are two
// 16-byte chunks (neighbours when interleaved, rot_dim / 2 dims apart otherwise), so
// a pair never leaves its lane; a warp works on four rows at a time. The 64 sines
// and cosines of a token are computed once per warp, two pairs a lane, handed round
// by shuffles, and used for all heads the warp takes. Four quads of rows per warp are on
// their way into shared memory, so that loads wait for no arithmetic, which is two lanes'
// floats an instruction.
//
// Bound by memory: 16384 tokens of 40 heads, normed and rotated, 52.2 us (6.43 TB/s read
// and written, 0.95 of a copy), of 80 heads with K and V on their way into the cache 102.8
// (6.53 TB/s, 0.96); 2047 tokens of 48 heads (7.4 us of bytes) 14.5, where a warp has a
// handful of quads; 4 tokens 2.4, a launch.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.h"
#include "rotary.h"
#include "rotary_split.h"

namespace pa {

__device__ int g_rotary_error;       // first device-side error of an append

namespace {

constexpr int kWarps = 4;
constexpr int kChunks = kHeadDim / 8;       // 16-byte chunks of a row
constexpr int kCtasPerSm = 6;
constexpr int kDepth = 4;                   // quads of rows a warp has on their way

// The 8 pairs (a, b) of a lane's two chunks, two pairs to a Two, and back. Interleaved pairs
// are the words of the chunks; otherwise a is the first chunk and b the second.
template <bool INTERLEAVED>
__device__ __forceinline__ void unpack(const uint4 (&w)[2], Two (&a)[4], Two (&b)[4]) {
    const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTERLEAVED) {
            a[i] = Two{bf16_lo(u[2 * i]), bf16_lo(u[2 * i + 1])};
            b[i] = Two{bf16_hi(u[2 * i]), bf16_hi(u[2 * i + 1])};
        } else {
            a[i] = Two{bf16_lo(u[i]), bf16_hi(u[i])};
            b[i] = Two{bf16_lo(u[i + 4]), bf16_hi(u[i + 4])};
        }
    }
}
template <bool INTERLEAVED>
__device__ __forceinline__ void pack(const Two (&a)[4], const Two (&b)[4], uint4 (&w)[2]) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTERLEAVED) {
            u[2 * i] = pack_bf16x2(a[i].x, b[i].x);
            u[2 * i + 1] = pack_bf16x2(a[i].y, b[i].y);
        } else {
            u[i] = pack_bf16x2(a[i].x, a[i].y);
            u[i + 4] = pack_bf16x2(b[i].x, b[i].y);
        }
    }
    w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    w[1] = make_uint4(u[4], u[5], u[6], u[7]);
}

template <bool APPEND, bool INTERLEAVED>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
rotate_kernel(const __grid_constant__ RotateArgs a) {
    __shared__ uint4 s_ring[kWarps][kDepth * 64];
    __shared__ uint64_t s_turns[kRotaryPairs];
    // weights in fp32, as the lanes hold a row: of q, of k; a and b; lane % 8
    __shared__ float4 s_weight[2][2][2][8];
    const int lane = threadIdx.x & 31, sub = lane & 7;
    // this lane's chunks of a row, and whether its pairs are rotated
    const bool rotated = sub * 8 < a.pairs;
    const bool apart = !INTERLEAVED && rotated;
    const int c0 = apart ? sub : 2 * sub, c1 = apart ? sub + a.pairs / 8 : 2 * sub + 1;
    const int hq = a.num_q_heads, hk = a.num_kv_heads, rows = hq + hk + (APPEND ? hk : 0);
    const unsigned items = a.num_tokens * a.slices, stride = gridDim.x * kWarps, slices = a.slices;
    const int quad_rows = a.quads * 4;
    // programmatic dependent of whatever precedes the call
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    // The warp's quads in order, kDepth - 1 of them on their way to shared memory while one is
    // worked on (held in registers, two of them, 24 warps kept the memory 60 % busy). A
    // lane copies what it reads itself.
    uint4 *ring = s_ring[threadIdx.x >> 5] + lane;
    unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5);
    unsigned item_ahead = item, t_ahead = item / slices;
    int h_ahead = (int)(item - t_ahead * slices) * quad_rows, end_ahead = min(h_ahead + quad_rows, rows), put = 0;
    auto fetch = [&]() {
        if (item_ahead < items) {
            const int h = h_ahead + (lane >> 3);
            if (h < end_ahead) {
                const HeadRows &r = h < hq ? a.q : (!APPEND || h < hq + hk ? a.k : a.v);
                const int64_t head = h < hq ? h : (!APPEND || h < hq + hk ? h - hq : h - hq - hk);
                const uint4 *src = r.p + t_ahead * r.token + head * r.head;
                const uint32_t dst = smem_u32(ring + put * 64);
                cp_async_16(dst, src + c0, 16);
                cp_async_16(dst + 512, src + c1, 16);
            }
            h_ahead += 4;
            if (h_ahead >= end_ahead) {
                item_ahead += stride;
                t_ahead = item_ahead / slices;
                h_ahead = (int)(item_ahead - t_ahead * slices) * quad_rows;
                end_ahead = min(h_ahead + quad_rows, rows);
            }
        }
        put = put + 1 == kDepth ? 0 : put + 1;
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kDepth - 1; ++i) fetch();
    for (int i = threadIdx.x; i < kRotaryPairs; i += kWarps * 32) s_turns[i] = a.turns[i];
    if (threadIdx.x < 16) {
        const int key = threadIdx.x >> 3;
        const uint4 *w = key ? a.k_weight : a.q_weight;
        if (w) {
            const uint4 x[2] = {__ldg(w + c0), __ldg(w + c1)};
            Two f[2][4];
            unpack<INTERLEAVED>(x, f[0], f[1]);
#pragma unroll
            for (int ab = 0; ab < 2; ++ab)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    s_weight[key][ab][i][sub] = make_float4(f[ab][2 * i].x, f[ab][2 * i].y, f[ab][2 * i + 1].x, f[ab][2 * i + 1].y);
        }
    }
    __syncthreads();
    int get = 0;
#pragma unroll 1
    for (; item < items; item += stride) {
        const int64_t t = item / slices;
        const int first = (int)(item - (unsigned)t * slices) * quad_rows, last = min(first + quad_rows, rows);
        // where the rows of q, k and v would begin if all were one's: row h of the token is
        // the h-th of its own from there on
        uint4 *const to_q = a.q_out.p + t * a.q_out.token;
        uint4 *to_k = a.k_out.p + t * a.k_out.token - hq * a.k_out.head, *to_v = nullptr;
        int64_t k_step = a.k_out.head;          // from a head's row to the next
        bool stored = true;
        if (APPEND) {
            const int64_t slot = __ldg(a.slots + t);
            stored = slot >= 0 && slot < a.num_slots;
            if (!stored && slot != -1 && lane == 0) atomicCAS(&g_rotary_error, 0, kErrBadSlot);
            const int lb = a.block_size_log2;
            const int64_t row = a.head_major ? ((slot >> lb) * hk << lb) + (slot & ((1 << lb) - 1)) : slot * hk;
            k_step = a.head_major ? kChunks << lb : kChunks;
            to_k = a.k_cache + row * kChunks - hq * k_step;
            to_v = a.v_cache + row * kChunks - (hq + hk) * k_step;
        }
        Two cs[4], sn[4];
        if (a.positions) {
            // pairs 2 lane and 2 lane + 1, then each lane the 8 of its own
            const int p = __ldg(a.positions + t);
            float c2[2], s2[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint64_t turn = (uint64_t)(int64_t)p * s_turns[2 * lane + k];
                sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s2[k], &c2[k]);
                s2[k] *= a.amplitude;
                c2[k] *= a.amplitude;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cs[j] = Two{__shfl_sync(0xffffffffu, c2[0], 4 * sub + j), __shfl_sync(0xffffffffu, c2[1], 4 * sub + j)};
                sn[j] = Two{__shfl_sync(0xffffffffu, s2[0], 4 * sub + j), __shfl_sync(0xffffffffu, s2[1], 4 * sub + j)};
            }
        }
#pragma unroll 1
        for (int h0 = first; h0 < last; h0 += 4) {
            fetch();
            cp_async_wait<kDepth - 1>();
            uint4 x[2] = {ring[get * 64], ring[get * 64 + 32]};
            get = get + 1 == kDepth ? 0 : get + 1;
            const int h = h0 + (lane >> 3);
            const bool key = h >= hq, value = APPEND && h >= hq + hk;
            const bool norm = !value && (key ? a.k_weight : a.q_weight) != nullptr;
            const bool turn = !value && rotated;
            Two f[4], g[4];
            unpack<INTERLEAVED>(x, f, g);
            Two sq = mul(f[0], f[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) sq = fma2(f[i], f[i], sq);
#pragma unroll
            for (int i = 0; i < 4; ++i) sq = fma2(g[i], g[i], sq);
            float sum = sq.x + sq.y;
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            if (norm) {
                const float inv = rsqrtf(fmaf(sum, 1.f / kHeadDim, a.eps));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 wa = s_weight[key][0][i][sub], wb = s_weight[key][1][i][sub];
                    f[2 * i] = mul(f[2 * i], mul(Two{wa.x, wa.y}, Two{inv, inv}));
                    f[2 * i + 1] = mul(f[2 * i + 1], mul(Two{wa.z, wa.w}, Two{inv, inv}));
                    g[2 * i] = mul(g[2 * i], mul(Two{wb.x, wb.y}, Two{inv, inv}));
                    g[2 * i + 1] = mul(g[2 * i + 1], mul(Two{wb.z, wb.w}, Two{inv, inv}));
                }
            }
            if (turn) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Two u = fma2(g[j], Two{-sn[j].x, -sn[j].y}, mul(f[j], cs[j]));
                    g[j] = fma2(f[j], sn[j], mul(g[j], cs[j]));
                    f[j] = u;
                }
            }
            // neither normed nor rotated: the bits as they are
            if (norm || turn) pack<INTERLEAVED>(f, g, x);
            if (h < last && (!key || stored)) {
                uint4 *out = !key ? to_q : (value ? to_v : to_k);
                out += h * (!key ? a.q_out.head : k_step);
                out[c0] = x[0];
                out[c1] = x[1];
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

namespace {

// radians / 2 pi in units of 2^-64 of a turn, modulo one turn, to the nearest: the 53 bits of a
// double times 1 / 2 pi to 128 bits behind the point, in whole numbers. (In doubles the
// quotient is off by 2^-54 of itself and more: at position 2^31 a frequency of 1 by 2^-25 turns,
// one of 2^20 by 2^-5.)
uint64_t turns_of(double radians) {
    constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;    // 2^128 / 2 pi
    int e;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(radians), &e), 53);    // |radians| = m 2^(e - 53)
    const unsigned __int128 lo = (unsigned __int128)m * kLo, hi = (unsigned __int128)m * kHi + (uint64_t)(lo >> 64);
    const uint64_t product[3] = {(uint64_t)lo, (uint64_t)hi, (uint64_t)(hi >> 64)};     // below 2^179
    auto word = [&](int i) { return i < 3 ? product[i] : 0; };
    const int shift = 53 + 128 - 64 - e;        // 96 and up: frequencies are 2^20 at most
    auto from_bit = [&](int b) {                // 64 bits of the product
        return word(b / 64) >> b % 64 | (b % 64 ? word(b / 64 + 1) << (64 - b % 64) : 0);
    };
    const uint64_t turns = from_bit(shift) + (from_bit(shift - 1) & 1);
    return radians < 0 ? 0 - turns : turns;
}

}  // namespace

void rotary_fill(pa_rotary_t *r, int rot_dim, int interleaved, const double *radians, double amplitude) {
    std::memset(r, 0, sizeof(*r));
    r->rot_dim = rot_dim;
    r->interleaved = interleaved ? 1 : 0;
    r->amplitude = (float)amplitude;
    for (int i = 0; i < rot_dim / 2; ++i) r->turns[i] = turns_of(radians[i]);
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
    const RotarySplit split = rotary_split(a.num_tokens, rows, sm_count);
    a.quads = split.quads;
    a.slices = split.slices;
    int64_t grid = (a.num_tokens * a.slices + kWarps - 1) / kWarps;
    if (grid > (int64_t)sm_count * kCtasPerSm * 3) grid = (int64_t)sm_count * kCtasPerSm * 3;
    if (append)
        return interleaved ? launch<true, true>(a, (unsigned)grid, stream)
                           : launch<true, false>(a, (unsigned)grid, stream);
    return interleaved ? launch<false, true>(a, (unsigned)grid, stream)
                       : launch<false, false>(a, (unsigned)grid, stream);
}

}  // namespace pa
