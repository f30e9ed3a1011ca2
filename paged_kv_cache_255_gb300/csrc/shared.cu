// Decode attention over shared prefixes, first half: for every group of
// sequences whose first blocks are the same, the attention of all its query
// rows to those blocks, computed once on the tensor cores.
//
// softmax over a sequence's keys splits into disjoint sets: with m, l, o the
// running max, sum of weights and weighted sum of V of a set, the sets of the
// prefix and of the sequence's own tokens merge by the usual log-sum-exp rule.
// Here the prefix's (m, l, o) are left in fp32 for every (sequence, query
// head); decode.cu folds them into each sequence's own part.
//
// The queries of a group against its prefix are a matrix product: n sequences
// x g heads rows per KV head against `tokens` keys, 4 n g tokens 128 flop per
// 512 bytes of K and V. Read per sequence the same prefix costs n times the
// bytes (from L2 at best) and n times the instructions: that bound the plain
// decode of 128 sequences x 8 heads over 2048 shared tokens (issue-bound at
// 97 us, with 143 MB of distinct rows that take 21 us to read).
//
//   plan kernel    one CTA: which tokens of each group are computed together
//                  (below), the active groups and the flat tile space.
//   prefix kernel  one CTA per SM. A unit is 256 query rows (two tiles of 128:
//                  128 / G sequences x G heads, G = g rounded up to a power of
//                  two) of one (group, KV head); its keys go in tiles of 128.
//                  The P CTAs take equal contiguous shares of the flat space of
//                  all units' key tiles, so any mix of groups fills the GPU;
//                  where every group has n pairs of tiles, n lanes of P / n
//                  CTAs each, so that the pairs of a KV head read the same
//                  keys at the same time. A unit that one CTA computes whole leaves its rows in unit_o,
//                  one that several share leaves a piece per CTA in part_o.
//                  Both are written [dim / 4][row] in 16-byte words, so a warp
//                  of rows writes 512 contiguous bytes.
//
// Tokens computed together: at most prefix_blocks * block_size, and at most the
// shortest non-empty length of the group's sequences rounded down to 16. So
// every key of the prefix is visible to every row that counts, no row is
// masked, and what a sequence must not see never enters its sums. Sequences of
// length 0 take no part (their rows are computed and dropped).
//
// The prefix kernel and the reading of the sequences' own tokens run at the same
// time on SMs of their own: one is bound by the tensor pipe and by the softmax
// between its products, the other by memory, and neither leaves room for the other
// on an SM. 128 sequences x 64 heads over 2048 shared and 256 own tokens:
// 39 to 44 us (pa_decode 86.5, the bytes alone 21.7), of which about 10 are the plan
// and the launches up to the first loads and 5 the combine. 256 x 32 over 32768
// shared and 16 .. 1000 own: 144 us (pa_decode 2198, the bytes alone 99); the 104
// SMs of the prefix keep their tensor pipes 66 % busy, a pair of 128-key products
// of both kinds taking 3230 cycles, the softmax of a tile 1275. (Times of calls here
// are of one within a graph of 20: the device's, without the host's.)
//
// Inside the prefix kernel (TMEM: S_A 0-127, O_A 128-255, S_B 256-383, O_B
// 384-511 columns; P_t in bf16 over the first 64 columns of S_t):
//   warps 0-3, 4-7   softmax of tile A, B: thread t owns row t (TMEM lane t)
//   warps 8, 9       K and V producers: a lane fetches one box of a block's
//                    tokens (16 .. 128) x 64 dims; the V warp also loads the
//                    queries
//   warp 10          issues S = Q K^T and O += P V as their inputs arrive
// Hand-offs are mbarriers; every wait is bounded (about 2 s), and a wait that
// ran out makes every role skip to its end. A role ends when what it has in
// flight has landed (or 0.1 s later); then the CTA frees its TMEM.
#include <climits>
#include <cmath>

#include "common.cuh"
#include "shared.h"
#include "tcgen05.cuh"

namespace pa {

__device__ int g_shared_error;       // first device-side error of a prefix launch

namespace {

constexpr int kPlanThreads = 256;      // 1024: 1.4 us more a call, every warp issuing every instruction
constexpr int kMaxGroups = kSharedMaxGroups;
constexpr int kRows = 128;                              // rows per query tile
constexpr int kKeys = 128;                              // keys per K/V tile
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kSoftmaxThreads = 256;
constexpr int kKWarp = kSoftmaxThreads / 32;             // 8
constexpr int kVWarp = kKWarp + 1;                       // 9
constexpr int kMmaWarp = kKWarp + 2;                     // 10
constexpr int kThreads = kSoftmaxThreads + 3 * 32;
constexpr int kGroup = 16;                               // tokens of the smallest TMA box, and per MMA of P V
constexpr int kGroups = kKeys / kGroup;                  // 8
constexpr uint32_t kQBytes = kRows * kRowBytes;         // 32 KB: 2 halves of [128][128 B]
constexpr uint32_t kQHalf = kRows * 128;
constexpr uint32_t kKVBytes = kKeys * kRowBytes;
constexpr uint32_t kKVHalf = kKeys * 128;
constexpr uint32_t kOffQ = 0;                           // Q_A, Q_B
constexpr uint32_t kOffK = kOffQ + 2 * kQBytes;
constexpr uint32_t kOffV = kOffK + kKStages * kKVBytes;
constexpr uint32_t kOffCtl = kOffV + kVStages * kKVBytes;
constexpr uint32_t kBarQFull = 0;
constexpr uint32_t kBarQEmpty = 1;
constexpr uint32_t kBarKFull = 2;                        // + stage
constexpr uint32_t kBarKEmpty = kBarKFull + kKStages;
constexpr uint32_t kBarVFull = kBarKEmpty + kKStages;
constexpr uint32_t kBarVEmpty = kBarVFull + kVStages;
constexpr uint32_t kBarSFull = kBarVEmpty + kVStages;    // + query tile (A 0, B 1)
constexpr uint32_t kBarPReady = kBarSFull + 2;
constexpr uint32_t kBarPVDone = kBarPReady + 2;
constexpr uint32_t kBarOFree = kBarPVDone + 2;
constexpr uint32_t kBarDrain = kBarOFree + 2;            // all products issued are done
constexpr uint32_t kNumBars = kBarDrain + 1;
constexpr uint32_t kOffTmemSlot = kOffCtl + 8 * kNumBars;
constexpr uint32_t kOffAbort = kOffTmemSlot + 4;
constexpr uint32_t kWalkBytes = 80;
constexpr uint32_t kOffWalk = (kOffAbort + 4 + 15) & ~15u;        // one Walk per warp
constexpr uint32_t kSmemBytes = kOffWalk + kWalkBytes * (kThreads / 32);
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescS = tc::idesc_bf16(128, kKeys, false);
constexpr uint32_t kIdescPV = tc::idesc_bf16(128, 128, true);
constexpr float kRescaleSlack = 8.f;                    // log2 units

__device__ __forceinline__ void set_error(int code) { atomicCAS(&g_shared_error, 0, code); }

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// Bounded wait that also gives up once the CTA's abort flag is set.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    for (;;) {
        if (tc::mbar_try_wait_sleep(bar, parity, 100000u)) return true;
        if (*abort) return false;
        if (tc::globaltimer_ns() - t0 > 2000000000ull) {
            set_error(kErrTimeout);
            *abort = 1;
            return false;
        }
    }
}

// Nothing a role has issued outlives it.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    if (!tc::drain_bar(bar, parity)) set_error(kErrTimeout);
}

// One lane waits for the warp; with `spin` the whole warp polls first (a
// suspended waiter resumes late).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                          bool spin = false) {
    if (spin) {
        for (int i = 0; i < 256; ++i)
            if (__any_sync(0xffffffffu, tc::mbar_test_wait(bar, parity))) {
                __syncwarp();
                return true;
            }
    }
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = wait_bar(bar, parity, abort);
    const bool r = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    __syncwarp();
    return r;
}
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void piece_end(SharedWalk &w) {
    const int64_t left = w.T1 - w.T;
    w.j1 = w.gr.nt - w.j0 < left ? w.gr.nt : w.j0 + (int)left;
}

// -- plan ------------------------------------------------------------------------

// Inclusive scans over the CTA's threads, several at once; `total` gets
// the sums over all threads. `sums` is scratch; the next call may follow at once.
template <int N, class T>
__device__ __forceinline__ void block_scan(T (&v)[N], T (&total)[N], T (*sums)[kPlanThreads / 32]) {
    constexpr int kWarps = kPlanThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const T n = __shfl_up_sync(0xffffffffu, v[k], off);
            if (lane >= off) v[k] += n;
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < N; ++k) sums[k][warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        T w = lane < kWarps ? sums[k][lane] : 0;
#pragma unroll
        for (int off = 1; off < kWarps; off <<= 1) {
            const T n = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += n;
        }
        total[k] = __shfl_sync(0xffffffffu, w, kWarps - 1);
        const T before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
        v[k] += warp > 0 ? before : 0;
    }
    __syncthreads();
}

// How a group's prefix is computed: not apart, by decode_shared_kernel for as
// many sequences at a time as fill the 8 columns of its tiles, or by
// shared_prefix_kernel.
enum Kind { kAlone, kPacked, kTensor };

// The cheapest, in SM time per KV head (us): 128 tokens take decode_shared_kernel
// 0.8 us for up to 8 columns (90 GB/s of K and V on an SM, once they are in L2);
// a key tile takes the prefix kernel 2 us for 256 rows, 1 when they fit one
// query tile, and every unit 4 us more. (12 prefixes of 3200 .. 9600 tokens for
// 5 sequences x 2 heads: 110 us packed, 79 on the prefix kernel; of 64 .. 768
// tokens: 25.0 packed, 28.4.)
__device__ __forceinline__ Kind cheapest(int live, int n, int tokens, int group, int group_pad,
                                         bool tensor_ok) {
    const int fit_log2 = shared_fit_log2(group), fit = 1 << fit_log2;
    const float len = (float)tokens * (1.f / kKeys);
    const float packed = 0.8f * len * (float)((n + fit - 1) >> fit_log2);
    const float pairs = (float)(((long long)n * group_pad + kPairRows - 1) / kPairRows);
    const float tensor = pairs * (4.f + ceilf(len) * (n * group_pad <= kRows ? 1.f : 2.f));
    if (live < kSharedMinSeqs || tokens == 0) return kAlone;
    if (tensor_ok && tensor < packed) return kTensor;
    return fit > 1 ? kPacked : kAlone;
}

// How many of the SMs compute the `tiles` prefix tiles of `units` units, while
// the others work through `own` 16-token tiles. Measured: a prefix tile pair
// takes about 1.6 us on an SM beside the other reads, a piece of a unit (its
// queries, first keys, last product and rows) 3 us more, and an SM reads up to
// 95 GB/s of K and V, all together 5.6 TB/s. SMs go to both in the proportion of
// the work, so that both end together. The pairs of a (group, KV head) should
// read the same keys at the same time, or the keys come from memory once for each:
// so the count is a multiple of the lanes, or with one lane a multiple of the units
// where the estimate is not a tenth worse. A multiple of the units also gives
// every SM one piece instead of two, and is taken where it is no worse. (SMs for
// the prefix and measured us: 256 sequences x 32 heads over 32768 and 16 .. 1000
// tokens, 4 lanes, 32 units: 96 158.8, 100 152.4, 104 146.1, 108 152.8, and in one lane 96 159,
// 100 185.6; 128 x 64 over 2048 and 256 tokens: 32 52.7, 52 45.5, 64 39.9, 72 42.3, 96 49.1.)
__device__ __forceinline__ int prefix_sms(int sm_count, float tiles, float units, float own, int lanes) {
    constexpr float kTile = 1.6f, kPiece = 3.f, kRate = 95e3f, kRateAll = 5.6e6f;
    const float sms = (float)sm_count, bytes = own * (2.f * kTileBytes);
    auto time = [&](float x, float pieces) {
        const float rate = fminf((sms - x) * kRate, kRateAll);
        return fmaxf(pieces * kPiece + ceilf(__fdividef(tiles, x)) * kTile, kPiece + __fdividef(bytes, rate));
    };
    // the prefix needs a SM microseconds, the rest b
    const float a = tiles * kTile + units * kPiece, b = bytes * (1.f / kRate) + 1.f;
    float best = fmaxf(1.f, fminf(floorf(__fdividef(sms * a, a + b) + 0.5f), sms - 1.f));
    best = fminf(best, tiles);
    float t = 1.1f;
    if (lanes > 1) {        // any multiple of the lanes will do
        const float step = (float)lanes;
        const float x = fminf(fmaxf(1.f, floorf(__fdividef(best, step) + 0.5f)), floorf(__fdividef(sms - 1.f, step))) * step;
        if (x >= 1.f && x <= tiles) {
            best = x;
            t = 1.f;
        }
    }
    t *= time(best, best >= tiles ? 1.f : 2.f + __fdividef(units, best));
    const float k = floorf(__fdividef(best, units));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float x = (k + (float)i) * units;
        const float u = x >= 1.f && x < sms && x <= tiles ? time(x, 1.f) : INFINITY;
        if (u <= t) {
            t = u;
            best = x;
        }
    }
    return (int)best;
}

__global__ void __launch_bounds__(kPlanThreads, 1)
shared_plan_kernel(const DecodeArgs a, const SharedArgs sh) {
    extern __shared__ int plan_smem[];
    __shared__ long long s_sums[1][kPlanThreads / 32];
    __shared__ int s_counts[3][kPlanThreads / 32];
    const int G = sh.num_groups, S = a.num_seqs, tid = threadIdx.x, lane = tid & 31;
    const int Hkv = a.num_kv_heads;
    const int fit_log2 = shared_fit_log2(a.group), fit = 1 << fit_log2;
    __shared__ int s_pairs;             // pairs of the first active group
    __shared__ bool s_differ;           // whether another has more or fewer
    __shared__ int s_packed[kPlanThreads];              // tokens of the first packed prefixes' entries
    int *bases = plan_smem;             // [G] flat index of the group's first tile
    int *starts = bases + G;            // [G + 1]
    int *tokens = starts + G + 1;       // [G] shortest non-empty length, then tokens computed together
    int *first = tokens + G;            // [G] first non-empty sequence, then first unit
    int *where = first + G;             // [G] non-empty sequences, then index of the active group or
                                        //     -2 - first entry of the packed prefix, or -1
    // programmatic dependent of whatever precedes the call
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int64_t max_len64 = (int64_t)a.max_blocks_per_seq << a.block_size_log2;
    const int max_len = (int)(max_len64 < INT_MAX ? max_len64 : INT_MAX);
    auto clamp = [](int x, int most) { return x < 0 ? 0 : (x > most ? most : x); };
    // the first of each input in flight together
    const int my_len = tid < S ? clamp(a.context_lens[tid], max_len) : 0;
    const int my_prefix = tid < G ? sh.prefix_blocks[tid] : 0;
    auto length = [&](int s) { return s == tid ? my_len : clamp(a.context_lens[s], max_len); };
    if (tid == 0) s_differ = false;
    for (int g = tid; g <= G; g += kPlanThreads) {
        starts[g] = clamp(sh.group_starts[g], S);
        if (g < G) {
            tokens[g] = first[g] = INT_MAX;
            where[g] = 0;
        }
    }
    __syncthreads();
    bool falls = false;
    for (int g = tid; g < G; g += kPlanThreads) falls |= starts[g] > starts[g + 1];
    const bool ordered = !__syncthreads_or(falls);     // else nothing is shared
    // the group of sequence s: the last one that starts at or before it
    auto group_of = [&](int s) {
        int lo = 0, hi = G;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid] <= s) lo = mid; else hi = mid;
        }
        return starts[lo] <= s && s < starts[lo + 1] ? lo : -1;
    };
    const int s_lo = starts[0], s_hi = starts[G];
    const int covered = s_hi > s_lo ? s_hi - s_lo : 0;
    int my_group = -1;                  // group of sequence tid
    for (int s0 = 0; s0 < s_hi; s0 += kPlanThreads) {
        const int s = s0 + tid;
        const int g = s < s_lo || s >= s_hi ? -1 : group_of(s);
        if (s0 == 0) my_group = g;
        const int L = g >= 0 ? length(s) : 0;
        const bool live = L > 0;
        // one atomic per warp where its sequences are of one group
        const int g0 = __shfl_sync(0xffffffffu, g, 0);
        if (__all_sync(0xffffffffu, g == g0)) {
            const int least = __reduce_min_sync(0xffffffffu, live ? L : INT_MAX);
            const unsigned m = __ballot_sync(0xffffffffu, live);
            if (m != 0 && lane == 0) {
                atomicMin(tokens + g0, least);
                atomicMin(first + g0, s + __ffs(m) - 1);
                atomicAdd(where + g0, __popc(m));
            }
        } else if (live) {
            atomicMin(tokens + g, L);
            atomicMin(first + g, s);
            atomicAdd(where + g, 1);
        }
    }
    __syncthreads();
    auto pairs_of = [&](int g) {
        return (int)(((int64_t)(starts[g + 1] - starts[g]) * sh.group_pad + kPairRows - 1) / kPairRows);
    };
    int base = 0, units = 0, act = 0, entries = covered;    // the host has ruled out 2^31 tiles
    for (int g0 = 0; g0 < G; g0 += kPlanThreads) {
        const int g = g0 + tid;
        SharedGroup gr{};
        Kind kind = kAlone;
        int chunks = 0;
        if (g < G) {
            const int64_t want = (int64_t)clamp(g0 == 0 ? my_prefix : sh.prefix_blocks[g], a.max_blocks_per_seq)
                                 << a.block_size_log2;
            const int most = where[g] > 0 ? tokens[g] & ~15 : 0;
            gr.tokens = (int)(want < most ? want : most);
            gr.row = first[g];
            gr.s0 = starts[g];
            gr.n = starts[g + 1] - starts[g];
            if (ordered) kind = cheapest(where[g], gr.n, gr.tokens, a.group, sh.group_pad, sh.tensor != 0);
            gr.nt = (gr.tokens + kKeys - 1) / kKeys;
            gr.pairs = pairs_of(g);
            if (kind == kPacked) chunks = (gr.n + fit - 1) >> fit_log2;
        }
        const bool tensor = kind == kTensor;
        const int u = tensor ? gr.pairs * Hkv : 0, tiles = u * gr.nt;
        // the active groups in the low 13 bits (kMaxGroups at most)
        int v[3] = {tiles, u, (chunks << 13) + tensor}, total[3];
        block_scan(v, total, s_counts);
        if (g < G) {
            gr.base = base + v[0] - tiles;
            gr.unit = units + v[1] - u;
            bases[g] = gr.base;
            first[g] = gr.unit;
            tokens[g] = kind == kAlone ? 0 : gr.tokens;
            where[g] = -1;
            if (tensor) {
                const int at = act + (v[2] & 0x1fff) - 1;
                where[g] = at;
                sh.groups[at] = gr;
                if (at == 0) s_pairs = gr.pairs;
            } else if (kind == kPacked) {
                const int at = entries + (v[2] >> 13) - chunks;
                where[g] = -2 - at;
                for (int c = 0; c < chunks; ++c) {
                    const int n = gr.n - c * fit < fit ? gr.n - c * fit : fit;
                    sh.entries[at + c] = SharedUnit{gr.row, gr.s0 + c * fit, 0, gr.tokens, n * a.group, 3, {0, 0}};
                    if (at + c - covered < kPlanThreads) s_packed[at + c - covered] = gr.tokens;
                }
            }
        }
        base += total[0];
        units += total[1];
        act += total[2] & 0x1fff;
        entries += total[2] >> 13;
    }
    __syncthreads();
    if (base > 0)
        for (int g = tid; g < G; g += kPlanThreads)
            if (where[g] >= 0 && pairs_of(g) != s_pairs) s_differ = true;     // read behind the scans below
    long long own = 0;
    for (int v0 = 0; v0 < entries; v0 += kPlanThreads) {
        const int v = v0 + tid;
        long long n[1] = {0}, total[1];
        if (v < covered) {
            const int s = s_lo + v;
            const int g = s == tid ? my_group : group_of(s), L = length(s);
            const int start = g >= 0 && L > 0 ? tokens[g] : 0;
            const int at = start > 0 ? where[g] : -1;
            const int nth = start > 0 ? s - starts[g] : 0;
            const int nth_row = nth * sh.group_pad;     // of the group's query rows
            sh.seq[s] = at <= -2 ? make_int4(-1, -2 - at + (nth >> fit_log2), (nth & (fit - 1)) * a.group, 0)
                        : at < 0 ? make_int4(-1, -1, 0, 0)
                                 : make_int4(first[g] + nth_row / kPairRows, -1, nth_row % kPairRows, pairs_of(g));
            sh.entries[v] = SharedUnit{s, s, start, L, a.group, start > 0 ? 1 : 0, {0, 0}};
            // an empty unit owns one (empty) tile
            n[0] = (L > start ? (L - start + kTileTokens - 1) / kTileTokens : 1) + kUnitTiles;
        } else if (v < entries) {
            const int p = v - covered;
            n[0] = (p < kPlanThreads ? s_packed[p] : sh.entries[v].len) / kTileTokens + kUnitTiles;
        }
        block_scan(n, total, s_sums);
        if (v < entries) sh.scan[v] = own + n[0];
        own += total[0];
    }
    own *= Hkv;
    const int sms = sh.max_workers, per_sm = a.num_workers / sms;
    int workers = 0, lanes = 1, tiles = 0, shares = 0;      // tiles and shares of a lane
    if (base > 0) {
        if (!s_differ) lanes = s_pairs;
        workers = prefix_sms(sms, (float)base, (float)units, (float)own, lanes);
        if (workers % lanes != 0) lanes = 1;    // fewer SMs than lanes
        tiles = base / lanes;
        shares = workers / lanes;
    }
    if (tid == 0) {
        SharedHeader h;
        h.tiles = tiles;
        h.lanes = lanes;
        h.shares = shares;
        h.own_tiles = own;
        h.s_lo = s_lo;
        h.s_hi = s_hi;
        h.entries = entries;
        h.workers = workers;
        const int64_t beside = (int64_t)(sms - workers) * per_sm, most = own / a.min_tiles;
        h.own_workers = (int)(most < 1 ? 1 : (most < beside ? most : beside));
        *sh.hdr = h;
    }
    // where each share begins: in the last group whose base is at or before its
    // first tile (groups without tiles share their successor's base, and come
    // before it)
    for (int w = tid; w < workers; w += kPlanThreads) {
        SharedWalk k{};
        k.lane = w % lanes;
        k.lanes = lanes;
        const int i = w / lanes;
        const int q = tiles / shares, r = tiles - q * shares;      // floor(i tiles / shares) in 32 bits
        k.T = i * q + i * r / shares;
        k.T1 = (i + 1) * q + (i + 1) * r / shares;
        const int at = (int)k.T * lanes;        // as if all lanes were one
        int lo = 0, hi = G;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (bases[mid] <= at) lo = mid; else hi = mid;
        }
        k.act = where[lo];
        k.gr = sh.groups[k.act];
        const int rem = (at - bases[lo]) / lanes, unit = rem / k.gr.nt, per_head = k.gr.pairs / lanes;
        k.j0 = rem - unit * k.gr.nt;
        k.kvh = unit / per_head;
        k.pair = k.lane + lanes * (unit - k.kvh * per_head);
        piece_end(k);
        sh.walks[w] = k;
    }
}

// -- prefix ------------------------------------------------------------------------

// Every warp walks by itself and keeps its place in shared memory, where the
// fields are read when they are needed: none stays live across the tile loop.
using Walk = SharedWalk;
static_assert(sizeof(Walk) == kWalkBytes, "SharedWalk");

// On to the next piece; false at the end of the share.
__device__ __forceinline__ bool walk_next(volatile Walk &place, const SharedArgs &sh, int num_kv_heads) {
    if (place.T + (place.j1 - place.j0) >= place.T1) return false;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        Walk &w = const_cast<Walk &>(place);
        w.T += w.j1 - w.j0;
        w.j0 = 0;
        w.pair += w.lanes;
        if (w.pair >= w.gr.pairs) {
            w.pair = w.lane;
            if (++w.kvh == num_kv_heads) {
                w.kvh = 0;
                w.gr = sh.groups[++w.act];
            }
        }
        piece_end(w);
    }
    __syncwarp();
    return true;
}

// Key tiles of a piece that a query tile (0 A, 1 B) computes: all, or none
// when the group's sequences end before the tile.
template <int G>
__device__ __forceinline__ int piece_tiles(const volatile Walk &w, int t) {
    return w.pair * (kPairRows / G) + t * (kRows / G) < w.gr.n ? w.j1 - w.j0 : 0;
}

// 16-token groups of key tile j that hold keys.
__device__ __forceinline__ int groups_used(const volatile Walk &w, int j) {
    const int n = (w.gr.tokens - j * kKeys) / kGroup;
    return n > kGroups ? kGroups : n;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
shared_prefix_kernel(const DecodeArgs a, const SharedArgs sh,
                     const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v,
                     const __grid_constant__ CUtensorMap tmap_q) {
    constexpr int BT = kRows / G;               // sequences per query tile
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5;
    // The SMs work in pairs that share a way to L2: a CTA whose neighbour streams own
    // tokens ended 13 us after the others (of 135). The first CTA starts beside the
    // plan's SM, which is still taken, and the next ones two by two: so it goes last.
    const int w_id = blockIdx.x == 0 ? (int)gridDim.x - 1 : (int)blockIdx.x - 1;
    if (tid == 0) {
        tc::prefetch_map(&tmap_k);
        tc::prefetch_map(&tmap_v);
        tc::prefetch_map(&tmap_q);
    }
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {                        // the swizzle atoms need 1024-byte alignment
        if (tid == 0) set_error(kErrSmemAlign);
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        return;
    }
    const uint32_t ctl = sbase + kOffCtl;
    auto bar = [&](uint32_t i) { return ctl + 8 * i; };
    volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffAbort);
    if (tid == 0) {
        tc::mbar_init(bar(kBarQFull), 1);
        tc::mbar_init(bar(kBarQEmpty), 1);
        for (int i = 0; i < kKStages; ++i) {
            tc::mbar_init(bar(kBarKFull + i), 1);
            tc::mbar_init(bar(kBarKEmpty + i), 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            tc::mbar_init(bar(kBarVFull + i), 1);
            tc::mbar_init(bar(kBarVEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(kBarSFull + i), 1);
            tc::mbar_init(bar(kBarPReady + i), kRows / 32);
            tc::mbar_init(bar(kBarPVDone + i), 1);
            tc::mbar_init(bar(kBarOFree + i), kRows / 32);
        }
        tc::mbar_init(bar(kBarDrain), 1);
        *abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) tc::tmem_alloc(sbase + kOffTmemSlot, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffTmemSlot);

    // the plan is complete before anything below reads it; the decode that
    // follows may be scheduled as this grid's CTAs finish
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    volatile Walk &w = reinterpret_cast<Walk *>(smem + kOffWalk)[warp];
    // the share's first piece together with the count of shares (a CTA without a
    // share reads what an earlier call left, and does not use it)
    if ((tid & 31) < (int)(sizeof(Walk) / 16))
        reinterpret_cast<int4 *>(smem + kOffWalk + warp * kWalkBytes)[tid & 31] =
            __ldcg(reinterpret_cast<const int4 *>(sh.walks + w_id) + (tid & 31));
    const bool works = w_id < __ldcg(&sh.hdr->workers);
    __syncwarp();
    if (!works) {
        // more CTAs than tiles
    } else if (tid < kSoftmaxThreads) {
        // ---------------- softmax warpgroups ----------------
        const int wg = tid >> 7, r = tid & 127;
        const uint32_t lane = (uint32_t)(r & ~31) << 16;
        const uint32_t tS = tmem + lane + wg * 256, tO = tS + 128;
        const float sc = a.scale_log2;          // above 0
        uint32_t gt = 0;                        // this query tile's key tiles before this piece
        bool ok = true;
        int piece = 0;
#pragma unroll 1
        do {
            const int ntt = piece_tiles<G>(w, wg);
            float m = -INFINITY, lsum = 0.f;
#pragma unroll 1
            for (int j = 0; j < ntt; ++j) {
                const uint32_t gj = gt + j;
                // S_t(j) done: also PV_t(j - 1), issued before it, so O is stable
                if (!warp_wait(bar(kBarSFull + wg), gj & 1, abort, true)) { ok = false; break; }
                tc::fence_after_sync();
                const int nkeys = w.gr.tokens - (w.j0 + j) * kKeys;     // keys from this tile on
                const bool need_mask = nkeys < kKeys;
                uint32_t sr[4][32];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) tc::tmem_ld32(tS + ch * 32, sr[ch]);
                tc::tmem_ld_wait();
                if (need_mask) {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (c >= nkeys - ch * 32) sr[ch][c] = 0xff800000u;     // -inf
                }
                // the largest raw score of the row, in four running values
                float e4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int c = 0; c < 32; c += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            e4[k] = fmax3(e4[k], __uint_as_float(sr[ch][c + 2 * k]),
                                          __uint_as_float(sr[ch][c + 2 * k + 1]));
                const float mt = fmax3(fmaxf(e4[0], e4[1]), e4[2], e4[3]) * sc;
                // the max is raised only when a tile exceeds it by 2^8: weights
                // stay below 2^8, far inside fp32 and bf16 range, and O is
                // rescaled rarely
                bool rescale = false;
                float alpha = 1.f;
                if (mt > m + kRescaleSlack) {
                    rescale = m != -INFINITY;
                    alpha = rescale ? ex2(m - mt) : 1.f;
                    lsum *= alpha;
                    m = mt;
                }
                const float mb = m == -INFINITY ? 0.f : m;
                // P = 2^(S sc - m), rounded to bf16 for the second product: its
                // error of 2^-9 per weight averages out over the keys, and the
                // output is rounded to bf16 as well
                float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t pw[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float p0 = ex2(fmaf(__uint_as_float(sr[ch][2 * c]), sc, -mb));
                        const float p1 = ex2(fmaf(__uint_as_float(sr[ch][2 * c + 1]), sc, -mb));
                        l4[c & 3] += p0 + p1;
                        pw[c] = pack_bf16x2(p0, p1);
                    }
                    tc::tmem_st16(tS + ch * 16, pw);
                }
                lsum += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t o[32];
                        tc::tmem_ld32(tO + ch * 32, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                        tc::tmem_st32(tO + ch * 32, o);
                    }
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                warp_arrive(bar(kBarPReady + wg));
            }
            if (!ok) break;
            if (ntt > 0) {
                if (!warp_wait(bar(kBarPVDone + wg), (gt + ntt - 1) & 1, abort, true)) { ok = false; break; }
                tc::fence_after_sync();
                // the row's (m, l) and unnormalised O in fp32: into the unit's
                // place when this share holds all its keys, else into a piece
                const int tok = w.pair * 2 * BT + wg * BT + r / G;
                const bool rv = tok < w.gr.n && r % G < a.group;
                const bool whole = w.j0 == 0 && w.j1 == w.gr.nt;
                const int64_t slot = 2 * w_id + (piece > 0 ? 1 : 0);
                const int64_t unit_rows = (int64_t)a.num_seqs * G;
                const int64_t row = whole ? (int64_t)(w.gr.s0 + tok) * G + r % G : wg * kRows + r;
                const int64_t stride = whole ? unit_rows : kPairRows;
                float4 *po = whole ? sh.unit_o + (int64_t)w.kvh * 32 * unit_rows : sh.part_o + slot * 32 * kPairRows;
                float2 *pml = whole ? sh.unit_ml + w.kvh * unit_rows : sh.part_ml + slot * kPairRows;
                if (rv) pml[row] = make_float2(m, lsum);
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t o[32];
                    tc::tmem_ld32(tO + ch * 32, o);
                    tc::tmem_ld_wait();
                    if (rv) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            po[(ch * 8 + c) * stride + row] =
                                make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                            __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
                    }
                }
            }
            tc::fence_before_sync();
            warp_arrive(bar(kBarOFree + wg));
            gt += ntt;
            ++piece;
        } while (walk_next(w, sh, a.num_kv_heads));
    } else if (warp == kKWarp || warp == kVWarp) {
        // ---------------- K and V producers ----------------
        const bool is_v = warp == kVWarp;
        const int nst = is_v ? kVStages : kKStages;
        const int lane = tid & 31;
        const int q = lane >> 1, h = lane & 1;      // this lane's box of a tile, and its half of the dims
        const int box = sh.box_tokens, boxes = kKeys / box;
        const void *map = is_v ? static_cast<const void *>(&tmap_v) : static_cast<const void *>(&tmap_k);
        const uint32_t bar_full = bar(is_v ? kBarVFull : kBarKFull);
        const uint32_t bar_empty = bar(is_v ? kBarVEmpty : kBarKEmpty);
        const uint32_t base = sbase + (is_v ? kOffV : kOffK);
        uint32_t gt = 0;                            // tiles issued
        int piece = 0, queries = 0;                 // pieces begun; pieces whose queries are issued
        bool ok = true;
#pragma unroll 1
        do {
            if (is_v) {
                // the queries, once the previous piece's MMAs are done with the buffers
                if (piece > 0 && !warp_wait(bar(kBarQEmpty), (piece - 1) & 1, abort)) { ok = false; break; }
                if (lane == 0) {
                    tc::mbar_expect_tx(bar(kBarQFull), 2 * kQBytes);
                    for (int t = 0; t < 2; ++t)
                        for (int hh = 0; hh < 2; ++hh)
                            tc::tma_load_3d(sbase + kOffQ + t * kQBytes + hh * kQHalf, &tmap_q, hh * 64,
                                            w.kvh * a.group, w.gr.s0 + w.pair * 2 * BT + t * BT, bar(kBarQFull));
                }
                warp_arrive(bar(kBarQFull));
                ++queries;
                if (lane == 0 && w.j0 == 0) {
                    // how the combine finds the unit: the shares from this one to the
                    // one of the unit's last key tile
                    const int64_t end = w.T + w.gr.nt;
                    const int parts = w.j1 == w.gr.nt ? 1
                                      : (int)((end * sh.hdr->shares - 1) / sh.hdr->tiles) - w_id / w.lanes + 1;
                    sh.parts[w.gr.unit + w.kvh * w.gr.pairs + w.pair] =
                        make_int4(2 * w_id + (piece > 0 ? 1 : 0), parts, 2 * w.lanes, 0);
                }
                __syncwarp();
            }
            // coordinates (dim 1, dim 2) of this lane's box of tile j; dim 1 (or
            // 2) at -kKeys reads zeros, for a block id outside the pool; x =
            // INT_MIN: no box. A box may reach past the prefix, but not past
            // its block: those keys are masked, their V not multiplied.
            auto box_at = [&](int j) -> int2 {
                const int t = j * kKeys + q * box;
                if (q >= boxes || j >= w.j1 || t >= w.gr.tokens) return make_int2(INT_MIN, 0);
                const int lb = a.block_size_log2;
                const int bid = __ldg(a.block_tables + (int64_t)w.gr.row * a.max_blocks_per_seq + (t >> lb));
                const int off = t & ((1 << lb) - 1);
                if (bid < 0 || (int64_t)bid >= a.num_blocks) {
                    set_error(kErrBadBlock);
                    return a.head_major ? make_int2(-kKeys, 0) : make_int2(w.kvh, -kKeys);
                }
                if (!a.head_major) return make_int2(w.kvh, (bid << lb) + off);
                return make_int2(off, bid * a.num_kv_heads + w.kvh);
            };
            int2 box_next = box_at(w.j0);
#pragma unroll 1
            for (int j = w.j0; j < w.j1; ++j) {
                const int2 at = box_next;
                box_next = box_at(j + 1);
                const int st = gt % nst;
                if (!warp_wait(bar_empty + 8 * st, ((gt / nst) & 1) ^ 1, abort)) { ok = false; break; }
                const uint32_t full = bar_full + 8 * st;
                const int n = __popc(__ballot_sync(0xffffffffu, at.x != INT_MIN));
                if (lane == 0) tc::mbar_expect_tx(full, (uint32_t)(n * box * 128));
                __syncwarp();
                if (at.x != INT_MIN)
                    tc::tma_load_3d(base + st * kKVBytes + h * kKVHalf + q * box * 128, map, h * 64, at.x, at.y, full);
                // the test hook holds back one V arrival (set_prefill_fault)
                if (!(is_v && sh.fault_hold_v && gt == 0)) warp_arrive(full);
                ++gt;
            }
            ++piece;
        } while (ok && walk_next(w, sh, a.num_kv_heads));
        // the last fill of every stage, and the last queries, have landed
        for (uint32_t g = gt > (uint32_t)nst ? gt - nst : 0; g < gt; ++g)
            drain(bar_full + 8 * (g % nst), (g / nst) & 1);
        if (queries > 0) drain(bar(kBarQFull), (queries - 1) & 1);
    } else if (warp == kMmaWarp) {
        // ---------------- MMA issue ----------------
        const uint64_t dq = tc::sw128_desc(sbase + kOffQ, 16, 1024);        // K-major
        const uint64_t dk = tc::sw128_desc(sbase + kOffK, 16, 1024);
        const uint64_t dv = tc::sw128_desc(sbase + kOffV, kKVHalf, 1024);   // MN-major: next 64 dims
        const uint32_t hi = (uint32_t)(dq >> 32);                           // same for all three
        const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
        auto desc = [hi](uint32_t lo) { return ((uint64_t)hi << 32) | lo; };
        auto issue_s = [&](int t, int st, uint32_t release) {
            const uint32_t qd = q_lo + t * (kQBytes >> 4);
            const uint32_t kd = k_lo + st * (kKVBytes >> 4);
            const uint32_t d = tmem + t * 256;
            tc::fence_after_sync();
            if (tc::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kHeadDim / 16; ++kk)
                    tc::mma_ss(d, desc(qd + (((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4)),
                               desc(kd + (((kk >> 2) * kKVHalf + (kk & 3) * 32) >> 4)), kIdescS, kk > 0);
                tc::commit(bar(kBarSFull + t));
                if (release) tc::commit(release);
            }
        };
        // over the first nv 16-key groups (the rest have P = 0 and no V)
        auto issue_pv = [&](int t, int st, bool acc, int nv, uint32_t release) {
            const uint32_t vd = v_lo + st * (kKVBytes >> 4);
            const uint32_t pa_ = tmem + t * 256;
            const uint32_t d = pa_ + 128;
            tc::fence_after_sync();
            if (tc::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kGroups; ++kk)
                    if (kk < nv)
                        tc::mma_ts(d, pa_ + kk * 8, desc(vd + ((kk * 2048) >> 4)), kIdescPV, acc || kk > 0);
                tc::commit(bar(kBarPVDone + t));
                if (release) tc::commit(release);
            }
        };
        // the warp polls, converged: the answer to every lane's test, bounded
        auto await = [&](uint32_t b, uint32_t parity) {
            uint64_t t0 = 0;
            for (uint32_t i = 0;; ++i) {
                if (__any_sync(0xffffffffu, tc::mbar_test_wait(b, parity))) {
                    __syncwarp();
                    return true;
                }
                if (i == 0) t0 = tc::globaltimer_ns();
                if ((i & 255) == 255) {
                    const bool stop = __shfl_sync(0xffffffffu,
                                                  (*abort || tc::globaltimer_ns() - t0 > 2000000000ull) ? 1 : 0, 0) != 0;
                    if (stop) {
                        if ((threadIdx.x & 31) == 0 && !*abort) {
                            set_error(kErrTimeout);
                            *abort = 1;
                        }
                        return false;
                    }
                }
            }
        };
        // In turn: PV_A(j), S_A(j + 1), PV_B(j), S_B(j + 1). PV_t(j) once P_t(j)
        // is in TMEM (and, for the first of a piece, the previous piece's O has
        // been read); the tiles it and S need have been waited for before, off
        // the chain from P to S. A stage is released after its last reader.
        uint32_t gt = 0, gq0 = 0, gq1 = 0;
        int piece = 0;
        bool ok = true;
#pragma unroll 1
        do {
            const int nt = w.j1 - w.j0;
            const bool two = piece_tiles<G>(w, 1) > 0;
            ok = await(bar(kBarQFull), piece & 1) && await(bar(kBarKFull + gt % kKStages), (gt / kKStages) & 1);
            if (ok) {
                issue_s(0, gt % kKStages, two ? 0u : bar(kBarKEmpty + gt % kKStages));
                if (two) issue_s(1, gt % kKStages, bar(kBarKEmpty + gt % kKStages));
            }
#pragma unroll 1
            for (int j = 0; ok && j < nt; ++j) {
                const uint32_t gp = gt + j, gs = gp + 1;
                const int vs = gp % kVStages, ks = gs % kKStages;
                const bool more = j + 1 < nt;
                const int nv = groups_used(w, w.j0 + j);
                ok = await(bar(kBarVFull + vs), (gp / kVStages) & 1);
                if (ok && more) ok = await(bar(kBarKFull + ks), (gs / kKStages) & 1);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t == 1 && !two) break;
                    const bool last = t == 1 || !two;
                    if (ok && j == 0 && piece > 0) ok = await(bar(kBarOFree + t), (piece - 1) & 1);
                    if (ok) ok = await(bar(kBarPReady + t), ((t == 0 ? gq0 : gq1) + j) & 1);
                    if (!ok) break;
                    issue_pv(t, vs, j > 0, nv, last ? bar(kBarVEmpty + vs) : 0u);
                    if (more) issue_s(t, ks, last ? bar(kBarKEmpty + ks) : 0u);
                }
            }
            // the queries' buffers are free once this piece's MMAs are done
            if (ok && tc::elect_one()) tc::commit(bar(kBarQEmpty));
            __syncwarp();
            gt += nt;
            gq0 += nt;
            gq1 += two ? nt : 0;
            ++piece;
        } while (ok && walk_next(w, sh, a.num_kv_heads));
        if (tc::elect_one()) tc::commit(bar(kBarDrain));
        __syncwarp();
        drain(bar(kBarDrain), 0);
    }

    // teardown: every role is done (or has given up) and has nothing in flight; TMEM is freed
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// q [S, Hq, 128] as (128, Hq, S) with boxes of 64 dims x G heads x 128 / G
// sequences: one half of a 128-row query tile.
bool make_q_map(CUtensorMap *m, const void *q, int num_seqs, int num_q_heads, int G) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)num_q_heads, (cuuint64_t)num_seqs};
    const cuuint64_t strides[2] = {(cuuint64_t)kRowBytes, (cuuint64_t)num_q_heads * kRowBytes};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kRows / G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_dependent(const void *fn, unsigned grid, unsigned block, size_t smem, void **args,
                             cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int G>
cudaError_t launch_g(const DecodeArgs &a, const SharedArgs &sh, cudaStream_t st) {
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void *>(&shared_prefix_kernel<G>), kSmemBytes);
    if (e != cudaSuccess) return e;
    const int bs = 1 << a.block_size_log2;
    CUtensorMap mk, mv, mq;
    if (!make_box_map(&mk, a.k_cache, a.num_blocks, bs, a.num_kv_heads, a.head_major != 0, sh.box_tokens) ||
        !make_box_map(&mv, a.v_cache, a.num_blocks, bs, a.num_kv_heads, a.head_major != 0, sh.box_tokens) ||
        !make_q_map(&mq, a.q, a.num_seqs, a.num_q_heads, G))
        return cudaErrorInvalidValue;
    DecodeArgs ac = a;
    SharedArgs sc = sh;
    void *args[] = {&ac, &sc, &mk, &mv, &mq};
    return launch_dependent(reinterpret_cast<const void *>(&shared_prefix_kernel<G>),
                            (unsigned)sh.max_workers, kThreads, kSmemBytes, args, st);
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Carve {
    size_t hdr, seq, entries, scan, groups, walks, parts, part_o, part_ml, unit_o, unit_ml, units, whole_o, whole_ml, end;
    Carve(int S, int G, int hq, int hkv, int gp, int workers) {
        const size_t rows = (size_t)S * gp * hkv, own = (size_t)S * hq, slots = 2 * (size_t)workers;
        hdr = 0;
        seq = hdr + round256(sizeof(SharedHeader));
        entries = seq + round256((size_t)S * sizeof(int4));
        scan = entries + round256(2 * (size_t)S * sizeof(SharedUnit));
        groups = scan + round256(2 * (size_t)S * sizeof(long long));
        walks = groups + round256((size_t)G * sizeof(SharedGroup));
        parts = walks + round256((size_t)workers * sizeof(SharedWalk));
        part_o = parts + round256((size_t)S * hkv * sizeof(int4));
        part_ml = part_o + slots * 32 * kPairRows * sizeof(float4);
        unit_o = part_ml + slots * kPairRows * sizeof(float2);
        unit_ml = unit_o + rows * 32 * sizeof(float4);
        units = unit_ml + round256(rows * sizeof(float2));
        whole_o = units + round256(2 * (size_t)S * hkv * sizeof(int4));
        whole_ml = whole_o + 2 * own * 32 * sizeof(float4);
        end = whole_ml + round256(2 * own * sizeof(float2));
    }
};

}  // namespace

cudaError_t take_shared_error(cudaStream_t stream, int *code) {
    return take_device_word(g_shared_error, stream, code);
}

size_t shared_workspace_bytes(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads,
                              int group_pad, int sm_count) {
    return Carve(num_seqs, num_groups, num_q_heads, num_kv_heads, group_pad, sm_count).end;
}

void shared_carve_workspace(SharedArgs &sh, void *workspace, const DecodeArgs &a) {
    const Carve c(a.num_seqs, sh.num_groups, a.num_q_heads, a.num_kv_heads, sh.group_pad, sh.max_workers);
    char *p = static_cast<char *>(workspace);
    sh.hdr = reinterpret_cast<SharedHeader *>(p + c.hdr);
    sh.seq = reinterpret_cast<int4 *>(p + c.seq);
    sh.entries = reinterpret_cast<SharedUnit *>(p + c.entries);
    sh.scan = reinterpret_cast<long long *>(p + c.scan);
    sh.groups = reinterpret_cast<SharedGroup *>(p + c.groups);
    sh.walks = reinterpret_cast<SharedWalk *>(p + c.walks);
    sh.parts = reinterpret_cast<int4 *>(p + c.parts);
    sh.part_o = reinterpret_cast<float4 *>(p + c.part_o);
    sh.part_ml = reinterpret_cast<float2 *>(p + c.part_ml);
    sh.unit_o = reinterpret_cast<float4 *>(p + c.unit_o);
    sh.unit_ml = reinterpret_cast<float2 *>(p + c.unit_ml);
    sh.units = reinterpret_cast<int4 *>(p + c.units);
    sh.whole_o = reinterpret_cast<float4 *>(p + c.whole_o);
    sh.whole_ml = reinterpret_cast<float2 *>(p + c.whole_ml);
}

cudaError_t launch_shared_prefix(const DecodeArgs &a, const SharedArgs &sh, cudaStream_t stream) {
    const size_t plan_smem = (5 * (size_t)sh.num_groups + 1) * sizeof(int);
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void *>(&shared_plan_kernel),
                                (int)((5 * kMaxGroups + 1) * sizeof(int)));
    if (e != cudaSuccess) return e;
    DecodeArgs ac = a;
    SharedArgs sc = sh;
    void *args[] = {&ac, &sc};
    e = launch_dependent(reinterpret_cast<const void *>(&shared_plan_kernel), 1, kPlanThreads, plan_smem,
                         args, stream);
    if (e != cudaSuccess) return e;
    if (!sh.tensor) return cudaSuccess;
    switch (sh.group_pad) {
        case 1: return launch_g<1>(a, sh, stream);
        case 2: return launch_g<2>(a, sh, stream);
        case 4: return launch_g<4>(a, sh, stream);
        case 8: return launch_g<8>(a, sh, stream);
        case 16: return launch_g<16>(a, sh, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
