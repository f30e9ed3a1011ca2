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
//                  all units' key tiles, so any mix of groups fills the GPU. A
//                  unit that one CTA computes whole leaves its rows in unit_o,
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
// Inside the prefix kernel (TMEM: S_A 0-127, O_A 128-255, S_B 256-383, O_B
// 384-511 columns; P_t in bf16 over the first 64 columns of S_t):
//   warps 0-3, 4-7   softmax of tile A, B: thread t owns row t (TMEM lane t)
//   warps 8, 9       K and V producers: 16 lanes fetch one box of 16 tokens x
//                    64 dims each; the V warp also loads the queries
//   warp 10          issues S = Q K^T and O += P V as their inputs arrive
// Hand-offs are mbarriers; every wait is bounded (about 2 s), and a wait that
// ran out makes every role skip to the end, where the CTA frees its TMEM.
#include <climits>
#include <cmath>

#include "common.cuh"
#include "shared.h"
#include "tcgen05.cuh"

namespace pa {

__device__ int g_shared_error;       // first device-side error of a prefix launch

namespace {

constexpr int kPlanThreads = 1024;
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
constexpr int kGroup = 16;                               // tokens per TMA box
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
constexpr uint32_t kNumBars = kBarOFree + 2;
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
__device__ __forceinline__ float fmin3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// Inclusive scan of v over the CTA's 1024 threads; `sums` is scratch of 32.
__device__ __forceinline__ long long block_scan(long long v, long long *sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long n = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += n;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    long long before = 0;
    for (int i = 0; i < warp; ++i) before += sums[i];
    return v + before;
}

// Estimated time (us) when x of the SMs compute `tiles` prefix tiles of `units`
// units and the others read `own` 16-token tiles at the same time. Measured: a
// prefix tile pair takes 2.3 us on an SM, 2.6 beside the other reads; a piece
// (its queries, first keys, last product and rows) 3 us; an SM reads 75 GB/s of
// K and V, and all together 6.4 TB/s. Equal shares of one group's units that
// end where units end have no piece more than they need. With x = all SMs the
// own tiles come after. Batch of 128 sequences x 64 heads, 2048 shared tokens
// and 256 own: x = 152, 88, 64, 40 took 65, 50, 48, 63 us.
__device__ __forceinline__ float split_cost(int x, int sms, long long tiles, long long units,
                                            long long own, bool one_group) {
    constexpr float kTile = 2.6f, kTileAlone = 2.3f, kPiece = 3.f, kRate = 75e3f, kRateAll = 6.4e6f;
    const float own_bytes = (float)own * (2.f * kTileBytes);
    const long long share = (tiles + x - 1) / x;
    const float nt = (float)tiles / (float)units;
    float pieces = 1.f + (float)share / nt;
    if (one_group && tiles % x == 0) {
        const long long n = tiles / units;
        if (n % share == 0) pieces = 1.f;
        else if (share % n == 0) pieces = (float)(share / n);
    }
    if (x == sms) return pieces * kPiece + (float)share * kTileAlone + own_bytes / kRateAll;
    const float rate = fminf((float)(sms - x) * kRate, kRateAll);
    return fmaxf(pieces * kPiece + (float)share * kTile, kPiece + own_bytes / rate);
}

__global__ void __launch_bounds__(kPlanThreads, 1)
shared_plan_kernel(const DecodeArgs a, const SharedArgs sh) {
    extern __shared__ long long plan_smem[];
    __shared__ long long s_sums[32];
    __shared__ unsigned long long s_best;
    const int G = sh.num_groups, S = a.num_seqs, tid = threadIdx.x;
    long long *bases = plan_smem;       // [G] flat index of the group's first tile
    int *starts = reinterpret_cast<int *>(bases + G);   // [G + 1]
    int *shortest = starts + G + 1;     // [G] shortest non-empty length, then tokens computed together
    int *first = shortest + G;          // [G] first non-empty sequence
    int *live = first + G;              // [G] non-empty sequences, then index among the active groups or -1
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
    for (int g = tid; g <= G; g += kPlanThreads) {
        starts[g] = clamp(sh.group_starts[g], S);
        if (g < G) {
            shortest[g] = first[g] = INT_MAX;
            live[g] = 0;
        }
    }
    __syncthreads();
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
    for (int s = tid; s < s_hi; s += kPlanThreads) {
        const int g = s < s_lo ? -1 : group_of(s), L = length(s);
        if (g >= 0 && L > 0) {
            atomicMin(shortest + g, L);
            atomicMin(first + g, s);
            atomicAdd(live + g, 1);
        }
    }
    __syncthreads();
    long long base = 0, units = 0;
    int act = 0;
    for (int g0 = 0; g0 < G; g0 += kPlanThreads) {
        const int g = g0 + tid;
        SharedGroup gr{};
        long long tiles = 0;
        if (g < G) {
            const int64_t want = (int64_t)clamp(g0 == 0 ? my_prefix : sh.prefix_blocks[g], a.max_blocks_per_seq)
                                 << a.block_size_log2;
            const int most = live[g] > 0 ? shortest[g] & ~15 : 0;
            gr.tokens = live[g] >= kSharedMinSeqs ? (int)(want < most ? want : most) : 0;
            gr.row = first[g];
            gr.s0 = starts[g];
            gr.n = starts[g + 1] - starts[g];
            gr.nt = (gr.tokens + kKeys - 1) / kKeys;
            gr.pairs = (int)(((int64_t)gr.n * sh.group_pad + kPairRows - 1) / kPairRows);
            tiles = (long long)gr.nt * gr.pairs * a.num_kv_heads;
        }
        const long long t_end = block_scan(tiles, s_sums);
        const long long u_end = block_scan(tiles > 0 ? ((long long)gr.pairs * a.num_kv_heads << 16) + 1 : 0, s_sums);
        const int a_end = (int)(u_end & 0xffff);        // at most kMaxGroups
        if (g < G) {
            const int at = act + a_end - 1;
            gr.base = base + t_end - tiles;
            bases[g] = gr.base;
            shortest[g] = gr.tokens;
            live[g] = tiles > 0 ? at : -1;
            if (tiles > 0) sh.groups[at] = gr;
        }
        __syncthreads();
        if (tid == kPlanThreads - 1) s_sums[0] = t_end, s_sums[1] = u_end;
        __syncthreads();
        base += s_sums[0];
        act += (int)(s_sums[1] & 0xffff);
        units += s_sums[1] >> 16;
        __syncthreads();
    }
    long long own = 0;
    for (int c0 = s_lo; c0 < s_hi; c0 += kPlanThreads) {
        const int s = c0 + tid;
        long long n = 0;
        if (s < s_hi) {
            const int g = group_of(s), L = length(s);
            const bool in = g >= 0 && live[g] >= 0 && L > 0;
            const int start = in ? shortest[g] : 0;
            sh.seq[s] = make_int2(start, in ? live[g] : -1);
            n = L > start ? (L - start + kTileTokens - 1) / kTileTokens : 1;   // an empty unit owns one tile
        }
        const long long end = block_scan(n, s_sums);
        if (s < s_hi) sh.scan[s] = own + end;
        __syncthreads();
        if (tid == kPlanThreads - 1) s_sums[0] = end;
        __syncthreads();
        own += s_sums[0];
        __syncthreads();
    }
    own *= a.num_kv_heads;
    // how many SMs compute prefixes while the others read the own tiles
    const int sms = sh.max_workers, per_sm = a.num_workers / sms;
    if (tid == 0) s_best = ~0ull;
    __syncthreads();
    for (int x = 1 + tid; x <= sms && x <= base; x += kPlanThreads) {
        const float cost = split_cost(x, sms, base, units, own, act == 1);
        atomicMin(&s_best, ((unsigned long long)__float_as_uint(cost) << 32) | (unsigned)x);
    }
    __syncthreads();
    const int workers = base > 0 ? (int)(s_best & 0xffffffffu) : 0;
    if (tid == 0) {
        SharedHeader h;
        h.tiles = base;
        h.own_tiles = own;
        h.s_lo = s_lo;
        h.s_hi = s_hi;
        h.workers = workers;
        const int64_t most = own / a.min_tiles;
        const int beside = workers < sms ? (sms - workers) * per_sm : a.num_workers;
        h.own_workers = (int)(most < 1 ? 1 : (most < beside ? most : beside));
        *sh.hdr = h;
    }
    // where each share begins: in the last group whose base is at or before its
    // first tile (groups without tiles share their successor's base, and come
    // before it)
    for (int w = tid; w < workers; w += kPlanThreads) {
        SharedWalk k{};
        k.T = (int64_t)w * base / workers;
        k.T1 = (int64_t)(w + 1) * base / workers;
        int lo = 0, hi = G;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (bases[mid] <= k.T) lo = mid; else hi = mid;
        }
        k.act = live[lo];
        k.gr = sh.groups[k.act];
        const int64_t rem = k.T - k.gr.base;
        const int unit = (int)(rem / k.gr.nt);
        k.j0 = (int)(rem - (int64_t)unit * k.gr.nt);
        k.kvh = unit / k.gr.pairs;
        k.pair = unit - k.kvh * k.gr.pairs;
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
        if (++w.pair == w.gr.pairs) {
            w.pair = 0;
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
    const int w_id = blockIdx.x;
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
    const bool works = w_id < sh.hdr->workers;
    if (works && (tid & 31) < (int)(sizeof(Walk) / 16))
        reinterpret_cast<int4 *>(smem + kOffWalk + warp * kWalkBytes)[tid & 31] =
            reinterpret_cast<const int4 *>(sh.walks + w_id)[tid & 31];
    __syncwarp();
    if (!works) {
        // more CTAs than tiles
    } else if (tid < kSoftmaxThreads) {
        // ---------------- softmax warpgroups ----------------
        const int wg = tid >> 7, r = tid & 127;
        const uint32_t lane = (uint32_t)(r & ~31) << 16;
        const uint32_t tS = tmem + lane + wg * 256, tO = tS + 128;
        const float sc = a.scale_log2;
        // loses against every score whatever the scale's sign
        const float masked = sc >= 0.f ? -INFINITY : INFINITY;
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
                            if (c >= nkeys - ch * 32) sr[ch][c] = __float_as_uint(masked);
                }
                // the extreme raw score of the row, in four running values
                float e4[4] = {masked, masked, masked, masked};
                if (sc >= 0.f) {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                        for (int c = 0; c < 32; c += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                e4[k] = fmax3(e4[k], __uint_as_float(sr[ch][c + 2 * k]),
                                              __uint_as_float(sr[ch][c + 2 * k + 1]));
                } else {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                        for (int c = 0; c < 32; c += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                e4[k] = fmin3(e4[k], __uint_as_float(sr[ch][c + 2 * k]),
                                              __uint_as_float(sr[ch][c + 2 * k + 1]));
                }
                const float ext = sc >= 0.f ? fmax3(fmaxf(e4[0], e4[1]), e4[2], e4[3])
                                            : fmin3(fminf(e4[0], e4[1]), e4[2], e4[3]);
                const float mt = ext == masked ? -INFINITY : ext * sc;
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
                        float p0 = ex2(fmaf(__uint_as_float(sr[ch][2 * c]), sc, -mb));
                        float p1 = ex2(fmaf(__uint_as_float(sr[ch][2 * c + 1]), sc, -mb));
                        if (need_mask) {
                            p0 = 2 * c < nkeys - ch * 32 ? p0 : 0.f;
                            p1 = 2 * c + 1 < nkeys - ch * 32 ? p1 : 0.f;
                        }
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
        const int q = lane >> 1, h = lane & 1;
        const void *map = is_v ? static_cast<const void *>(&tmap_v) : static_cast<const void *>(&tmap_k);
        const uint32_t bar_full = bar(is_v ? kBarVFull : kBarKFull);
        const uint32_t bar_empty = bar(is_v ? kBarVEmpty : kBarKEmpty);
        const uint32_t base = sbase + (is_v ? kOffV : kOffK);
        uint32_t gt = 0;
        int piece = 0;
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
            }
            // coordinates (dim 1, dim 2) of this lane's box of tile j; dim 1 (or
            // 2) at -kGroup reads zeros, for a block id outside the pool; x =
            // INT_MIN: no box
            auto box_at = [&](int j) -> int2 {
                if (lane >= 2 * kGroups || j >= w.j1 || q >= groups_used(w, j)) return make_int2(INT_MIN, 0);
                const int t = j * kKeys + q * kGroup;
                const int lb = a.block_size_log2;
                const int bid = __ldg(a.block_tables + (int64_t)w.gr.row * a.max_blocks_per_seq + (t >> lb));
                const int off = t & ((1 << lb) - 1);
                if (bid < 0 || (int64_t)bid >= a.num_blocks) {
                    set_error(kErrBadBlock);
                    return a.head_major ? make_int2(-kGroup, 0) : make_int2(w.kvh, -kGroup);
                }
                if (!a.head_major) return make_int2(w.kvh, (bid << lb) + off);
                return make_int2(off, bid * a.num_kv_heads + w.kvh);
            };
            int2 box_next = box_at(w.j0);
#pragma unroll 1
            for (int j = w.j0; j < w.j1; ++j) {
                const int2 box = box_next;
                box_next = box_at(j + 1);
                const uint32_t gj = gt + (j - w.j0);
                const int st = gj % nst;
                if (!warp_wait(bar_empty + 8 * st, ((gj / nst) & 1) ^ 1, abort)) { ok = false; break; }
                const uint32_t full = bar_full + 8 * st;
                if (lane == 0) tc::mbar_expect_tx(full, (uint32_t)groups_used(w, j) * 2 * kGroup * 128);
                __syncwarp();
                if (box.x != INT_MIN)
                    tc::tma_load_3d(base + st * kKVBytes + h * kKVHalf + q * kGroup * 128, map, h * 64, box.x,
                                    box.y, full);
                warp_arrive(full);
            }
            gt += w.j1 - w.j0;
            ++piece;
        } while (ok && walk_next(w, sh, a.num_kv_heads));
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
        auto ready = [](uint32_t b, uint32_t parity) {
            const bool r = __any_sync(0xffffffffu, tc::mbar_test_wait(b, parity));
            if (r) __syncwarp();
            return r;
        };
        // S_t(x) once K_x has landed and PV_t(x - 1) has been issued; PV_t(y)
        // once P_t(y) is in TMEM and V_y has landed (and, for the first of a
        // piece, the previous piece's O has been read). A stage is released
        // after its last reader.
        uint32_t gt = 0, gq0 = 0, gq1 = 0;
        int piece = 0;
        bool ok = true;
#pragma unroll 1
        do {
            const int nta = piece_tiles<G>(w, 0), ntb = piece_tiles<G>(w, 1);
            ok = warp_wait(bar(kBarQFull), piece & 1, abort);
            int sj0 = 0, sj1 = 0, pj0 = 0, pj1 = 0;     // next S / PV tile of A, B
            uint64_t t_idle = 0;
            uint32_t idle = 0;
#pragma unroll 1
            while (ok && (pj0 < nta || pj1 < ntb)) {
                bool progress = false;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    int &sj = t == 0 ? sj0 : sj1;
                    int &pj = t == 0 ? pj0 : pj1;
                    const int other_pj = t == 0 ? pj1 : pj0;
                    const int other_sj = t == 0 ? sj1 : sj0;
                    const int my_nt = t == 0 ? nta : ntb;
                    const int other_nt = t == 0 ? ntb : nta;
                    const uint32_t my_gq = t == 0 ? gq0 : gq1;
                    if (pj < sj) {
                        const uint32_t gp = gt + pj;
                        const int st = gp % kVStages;
                        bool go = ready(bar(kBarPReady + t), (my_gq + pj) & 1) &&
                                  ready(bar(kBarVFull + st), (gp / kVStages) & 1);
                        if (go && pj == 0 && piece > 0) go = ready(bar(kBarOFree + t), (piece - 1) & 1);
                        if (go) {
                            issue_pv(t, st, pj > 0, groups_used(w, w.j0 + pj),
                                     other_pj > pj || other_nt <= pj ? bar(kBarVEmpty + st) : 0u);
                            ++pj;
                            progress = true;
                        }
                    }
                    if (sj == pj && sj < my_nt) {
                        const uint32_t gs = gt + sj;
                        const int st = gs % kKStages;
                        if (ready(bar(kBarKFull + st), (gs / kKStages) & 1)) {
                            issue_s(t, st, other_sj > sj || other_nt <= sj ? bar(kBarKEmpty + st) : 0u);
                            ++sj;
                            progress = true;
                        }
                    }
                }
                if (progress) {
                    idle = 0;
                    continue;
                }
                if (++idle == 1) {
                    t_idle = tc::globaltimer_ns();
                } else if ((idle & 255) == 0) {
                    const bool stop = __shfl_sync(0xffffffffu,
                                                  (*abort || tc::globaltimer_ns() - t_idle > 2000000000ull) ? 1 : 0, 0) != 0;
                    if (stop) {
                        if ((threadIdx.x & 31) == 0 && !*abort) {
                            set_error(kErrTimeout);
                            *abort = 1;
                        }
                        ok = false;
                    }
                }
            }
            // the queries' buffers are free once this piece's MMAs are done
            if (tc::elect_one()) tc::commit(bar(kBarQEmpty));
            __syncwarp();
            gt += w.j1 - w.j0;
            gq0 += nta;
            gq1 += ntb;
            ++piece;
        } while (ok && walk_next(w, sh, a.num_kv_heads));
    }

    // teardown: every role is done (or has given up); TMEM is freed
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
    cudaError_t e = cudaFuncSetAttribute(shared_prefix_kernel<G>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    const int bs = 1 << a.block_size_log2;
    CUtensorMap mk, mv, mq;
    if (!make_pool_map(&mk, a.k_cache, a.num_blocks, bs, a.num_kv_heads, a.head_major != 0) ||
        !make_pool_map(&mv, a.v_cache, a.num_blocks, bs, a.num_kv_heads, a.head_major != 0) ||
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
    size_t hdr, seq, scan, groups, walks, part_o, part_ml, unit_o, unit_ml, units, own_o, own_ml, end;
    Carve(int S, int G, int hq, int hkv, int gp, int workers) {
        const size_t rows = (size_t)S * gp * hkv, own = (size_t)S * hq, slots = 2 * (size_t)workers;
        hdr = 0;
        seq = hdr + round256(sizeof(SharedHeader));
        scan = seq + round256((size_t)S * sizeof(int2));
        groups = scan + round256((size_t)S * sizeof(long long));
        walks = groups + round256((size_t)G * sizeof(SharedGroup));
        part_o = walks + round256((size_t)workers * sizeof(SharedWalk));
        part_ml = part_o + slots * 32 * kPairRows * sizeof(float4);
        unit_o = part_ml + slots * kPairRows * sizeof(float2);
        unit_ml = unit_o + rows * 32 * sizeof(float4);
        units = unit_ml + round256(rows * sizeof(float2));
        own_o = units + round256((size_t)S * hkv * sizeof(int4));
        own_ml = own_o + own * 32 * sizeof(float4);
        end = own_ml + round256(own * sizeof(float2));
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
    sh.seq = reinterpret_cast<int2 *>(p + c.seq);
    sh.scan = reinterpret_cast<long long *>(p + c.scan);
    sh.groups = reinterpret_cast<SharedGroup *>(p + c.groups);
    sh.walks = reinterpret_cast<SharedWalk *>(p + c.walks);
    sh.part_o = reinterpret_cast<float4 *>(p + c.part_o);
    sh.part_ml = reinterpret_cast<float2 *>(p + c.part_ml);
    sh.unit_o = reinterpret_cast<float4 *>(p + c.unit_o);
    sh.unit_ml = reinterpret_cast<float2 *>(p + c.unit_ml);
    sh.units = reinterpret_cast<int4 *>(p + c.units);
    sh.own_o = reinterpret_cast<float4 *>(p + c.own_o);
    sh.own_ml = reinterpret_cast<float2 *>(p + c.own_ml);
}

cudaError_t launch_shared_prefix(const DecodeArgs &a, const SharedArgs &sh, cudaStream_t stream) {
    const size_t plan_smem = (6 * (size_t)sh.num_groups + 1) * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(shared_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)((6 * kMaxGroups + 1) * sizeof(int)));
    if (e != cudaSuccess) return e;
    DecodeArgs ac = a;
    SharedArgs sc = sh;
    void *args[] = {&ac, &sc};
    e = launch_dependent(reinterpret_cast<const void *>(&shared_plan_kernel), 1, kPlanThreads, plan_smem,
                         args, stream);
    if (e != cudaSuccess) return e;
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
