// Decode attention over trees of drafted tokens: the n nodes of a sequence are the
// last n of its cached tokens; query row i sees everything before them and the nodes
// whose bits its mask sets ("Implementation Details", Speculative Decoding -- EAGLE
// Proposer: drafted tokens are verified by the target model).
//
//   out_i = sum_t softmax_t(scale q_i . K_t) V_t,  t < L - n or bit t - (L - n) of mask_i
//
// All rows of a sequence see the same long context, so n nodes x g heads of the KV
// head are the rows of one matrix product against its keys: K and V are read once
// for up to 256 of them. 4 n g 128 flop per 512 bytes of K and V: memory-bound up to
// n g = 128, and near the balance point above.
//
// A unit is 256 query rows (two tiles of 128: 128 / G tokens x G heads, G = g rounded up
// to a power of two) of one (sequence, KV head); its keys go in tiles of 128. The flat
// space of all units' key tiles, and kUnitPlaces places more a unit for what it costs
// besides them, is cut into equal contiguous shares, one CTA per SM each (but for what
// side by side lanes leave over: tree_lanes), planned by every CTA from the lengths and
// starts. A unit that one share holds whole is written
// as it ends; one that several share leaves a part per share in fp32, and
// tree_combine_kernel merges them by their running maxima and sums.
//
// Inside a CTA (TMEM: S_A 0-127, O_A 128-255, S_B 256-383, O_B 384-511 columns;
// P_t in bf16 over the first 64 columns of S_t):
//   warps 0-3, 4-7   softmax of stream A, B. Two query tiles are a stream each; the even
//                    and the odd key tiles of one query tile otherwise. Of more than 64
//                    rows thread t owns row t (TMEM lane t); up to 64 rows (32) stand 16
//                    (8) to a warp, a quad of lanes owning two rows (one), so that all four
//                    schedulers work and each for a half (a quarter) of the time.
//                    The mask's bits are read only on tiles that reach the nodes, and the V
//                    of those is cleaned by the same warps before its product: rows past
//                    the last token become 0, and so do infinities and NaN in nodes' rows (a
//                    weight of 0 times them is not 0). The rows that do see such a node add
//                    what was taken out after their result is written.
//   warps 8, 9       K and V producers: TMA boxes of a block's tokens (16 .. 128) x 64
//                    dims; the V warp also loads the queries
//   warp 10          issues S = Q K^T and O += P V as their inputs arrive
// Measured (calls in a graph, both kernels): 8 contexts of 32k to 131k tokens, up to 128 rows
// a unit, 406 - 425 us, 6.4 - 6.6 TB/s of 6.79: bound by memory. 512 units of 192 to 256 rows
// over 16 to 64 key tiles 258 - 281 us, 1110 - 1200 TFLOP/s of 1939: the tensor pipe is busy for
// 61 % of the cycles. A step's products take 2 x (512 + 512) cycles alone, about 1400 a query
// tile beside the other stream's TMEM traffic and the tiles' arrival (a product from shared memory
// reads 128 B a cycle, all there is), and a stream's chain P -> PV -> S -> P is 2700. 480 units of
// 1 to 8 tiles 42.1 us, where the floor is 21: 3 us until the plan is made, then 5 per unit
// of dependent steps (tiles, S, softmax, PV, result), and 3 for the merge. A softmax with a
// polynomial for a part of its powers of two is slower (a quarter of them: 319 us against 304):
// the XU pipe is busy for 28 %.
//
// Hand-offs are mbarriers; every wait is bounded (about 2 s), and a wait that ran out
// makes every role skip to its end. A role ends when what it has in flight has landed
// (or 0.1 s later); then the CTA frees its TMEM.
#include <climits>
#include <cmath>

#include "common.cuh"
#include "shared.h"
#include "tcgen05.cuh"
#include "tree.h"
#include "tree_plan.h"

namespace pa {

__device__ int g_tree_error;         // first device-side error of a launch

namespace {

constexpr int kRows = 128;                              // rows per query tile
constexpr int kPair = 2 * kRows;
constexpr int kKeys = kTreeKeys;                        // keys per K/V tile
static_assert(kPair == kTreePairRows && kKeys == 128, "two tiles of 128 rows, tiles of 128 keys");
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kSoftmaxThreads = 256;
constexpr int kKWarp = kSoftmaxThreads / 32;            // 8
constexpr int kVWarp = kKWarp + 1;                      // 9
constexpr int kMmaWarp = kKWarp + 2;                    // 10
constexpr int kThreads = kSoftmaxThreads + 3 * 32;
constexpr int kWarpsAll = kThreads / 32;
constexpr int kGroup = 16;                              // tokens per MMA of P V
constexpr int kGroups = kKeys / kGroup;                 // 8
constexpr int kCombineRows = 8;                         // rows merged at a time
// Places of a unit besides its tiles, for its start and its end: at 0, 1, 2, 3, 4 a batch of 512
// units of 16 to 64 tiles takes 275, 270, 267, 261, 261 us, 480 units of 1 to 8 tiles 53.3,
// 45.3, 41.8, 42.1, 43.2, a few small units 10.85, 11.0, 10.9, 10.8, 11.1, and 64 units of 256 to
// 1024 tiles 413 at each.
constexpr int kUnitPlaces = kTreeUnitPlaces;
constexpr uint32_t kQBytes = kRows * kRowBytes;         // 32 KB: 2 halves of [128][128 B]
constexpr uint32_t kQHalf = kRows * 128;
constexpr uint32_t kKVBytes = kKeys * kRowBytes;
constexpr uint32_t kKVHalf = kKeys * 128;
constexpr uint32_t kOffQ = 0;                           // Q_A, Q_B
constexpr uint32_t kOffK = kOffQ + 2 * kQBytes;
constexpr uint32_t kOffV = kOffK + kKStages * kKVBytes;
constexpr uint32_t kOffCtl = kOffV + kVStages * kKVBytes;
constexpr uint32_t kBarQFull = 0;                        // + buffer
constexpr uint32_t kBarQEmpty = 2;                       // + buffer
constexpr uint32_t kBarKFull = 4;                        // + stage
constexpr uint32_t kBarKEmpty = kBarKFull + kKStages;
constexpr uint32_t kBarVFull = kBarKEmpty + kKStages;
constexpr uint32_t kBarVEmpty = kBarVFull + kVStages;
constexpr uint32_t kBarSFull = kBarVEmpty + kVStages;    // + stream (A 0, B 1)
constexpr uint32_t kBarPReady = kBarSFull + 2;
constexpr uint32_t kBarPVDone = kBarPReady + 2;
constexpr uint32_t kBarOFree = kBarPVDone + 2;           // a piece's results are read
constexpr uint32_t kBarHalves = kBarOFree + 1;           // both streams' maxima and sums are there
constexpr uint32_t kBarDrain = kBarHalves + 1;           // all products issued are done
constexpr uint32_t kNumBars = kBarDrain + 1;
constexpr uint32_t kOffTmemSlot = kOffCtl + 8 * kNumBars;
constexpr uint32_t kOffAbort = kOffTmemSlot + 4;
constexpr uint32_t kWalkBytes = 56;
constexpr uint32_t kOffWalk = (kOffAbort + 4 + 15) & ~15u;        // one Walk per warp, and the plan's
constexpr int kOddSets = 4;                                       // of the pieces in flight: bit i, nodes 32 i ..
constexpr uint32_t kOffOdd = kOffWalk + kWalkBytes * (kWarpsAll + 1);   // 32 i + 31 have V that is not finite
constexpr uint32_t kOffHalves = kOffOdd + 4 * kOddSets;           // [2][128] float2; before that the plan's sums
constexpr uint32_t kSmemBytes = kOffHalves + 2 * kRows * 8;
static_assert(kOffHalves % 8 == 0, "pairs of floats, and a 64-bit count");
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescS = tc::idesc_bf16(128, kKeys, false);
constexpr uint32_t kIdescPV = tc::idesc_bf16(128, 128, true);
constexpr uint32_t kNegateA = 1u << 13;                 // of an instruction descriptor
constexpr uint32_t kMasked = 0xff800000u;               // -infinity
constexpr float kRescaleSlack = 8.f;                    // log2 units

__device__ __forceinline__ void set_error(int code) { atomicCAS(&g_tree_error, 0, code); }

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// The kernel's code has to stay small: at 200 KB every unit's straight-line code came from
// L2 again (an epilogue of 16 stores took 7000 cycles). What runs once a piece or
// less is therefore out of line.

// Bounded wait that also gives up once the CTA's abort flag is set.
__device__ __noinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort) {
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
__device__ __noinline__ void drain(uint32_t bar, uint32_t parity) {
    if (!tc::drain_bar(bar, parity)) set_error(kErrTimeout);
}

// The warp polls, converged: the answer to every lane's test (a suspended waiter resumes
// late), bounded; without `spin` one lane waits for it.
__device__ __noinline__ bool warp_wait_more(uint32_t bar, uint32_t parity, volatile int *abort, bool spin) {
    if (spin) {
        const uint64_t t0 = tc::globaltimer_ns();
#pragma unroll 1
        for (uint32_t i = 1;; ++i) {
            if (__any_sync(0xffffffffu, tc::mbar_test_wait(bar, parity))) break;
            if ((i & 255) == 0) {
                const bool late = tc::globaltimer_ns() - t0 > 2000000000ull;
                if (__any_sync(0xffffffffu, late || *abort)) {
                    if ((threadIdx.x & 31) == 0 && !*abort) {
                        set_error(kErrTimeout);
                        *abort = 1;
                    }
                    return false;
                }
            }
        }
        __syncwarp();
        return true;
    }
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = wait_bar(bar, parity, abort);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    __syncwarp();
    return ok;
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, bool spin = false) {
    if (__any_sync(0xffffffffu, tc::mbar_test_wait(bar, parity))) {
        __syncwarp();
        return true;
    }
    return warp_wait_more(bar, parity, abort, spin);
}
// One lane's wait.
__device__ __noinline__ bool lane_wait_more(uint32_t bar, uint32_t parity, volatile int *abort) {
    const uint64_t t0 = tc::globaltimer_ns();
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (tc::mbar_test_wait(bar, parity)) return true;
        if ((i & 255) == 0) {
            if (*abort) return false;
            if (tc::globaltimer_ns() - t0 > 2000000000ull) {
                set_error(kErrTimeout);
                *abort = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    return tc::mbar_test_wait(bar, parity) || lane_wait_more(bar, parity, abort);
}
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// -- plan ------------------------------------------------------------------------

using Seq = TreeSeq;

template <int G>
__device__ __noinline__ Seq load_seq(const TreeArgs &a, int s) {
    const int64_t max_len = (int64_t)a.max_blocks_per_seq << a.block_size_log2;     // below 2^31
    return tree_seq(__ldg(a.starts + s), __ldg(a.starts + s + 1), __ldg(a.context_lens + s), a.total_q, max_len, G);
}

// A share's walk over the flat space of its lane, sequence by sequence, KV head, pair, key
// tile: its pieces are runs of key tiles [j0, j1) of one unit. Every warp walks by itself
// and keeps its place in shared memory, where the fields are read when they are needed:
// none stays live across the tile loop.
struct Walk {
    int T, T1;          // place of tile j0, end of the share
    Seq q;
    int s, kvh, pair, j0, j1;
    int lane, lanes;
};
static_assert(sizeof(Walk) == kWalkBytes, "Walk");

__device__ __forceinline__ void piece_end(Walk &w) {
    const int left = w.T1 - w.T;
    w.j1 = w.q.nt - w.j0 < left ? w.q.nt : w.j0 + left;
}

// On to the next unit; false at the end of the share.
template <int G>
__device__ __noinline__ bool next_unit(Walk &w, const TreeArgs &a) {
    w.T += w.q.nt - w.j0 + kUnitPlaces;
    if (w.T >= w.T1) return false;
    w.j0 = 0;
    w.pair += w.lanes;
    if (w.pair >= w.q.pairs) {
        w.pair = w.lane;
        if (++w.kvh == a.num_kv_heads) {
            w.kvh = 0;
            do w.q = load_seq<G>(a, ++w.s);         // the places left are some sequence's
            while (w.q.pairs == 0 && w.s + 1 < a.num_seqs);
        }
    }
    piece_end(w);
    return true;
}

template <int G>
__device__ __noinline__ bool walk_next(volatile Walk &place, const TreeArgs &a) {
    bool more = false;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) more = next_unit<G>(const_cast<Walk &>(place), a);
    more = __shfl_sync(0xffffffffu, more ? 1 : 0, 0) != 0;
    __syncwarp();
    return more;
}

// Where share i of `shares` begins among W places: floor(i W / shares). Both factors of the
// second term are below 256: half a unit, 1 / 512 of a share, is more than its quotient in
// fp32 is off by.
__device__ __forceinline__ int share_begin(int i, int W, int shares) {
    const int each = W / shares;
    return i * each + (int)__fdividef((float)(i * (W - each * shares)) + 0.5f, (float)shares);
}

// The share that place T is in: a guess, which is off by one at most.
__device__ __forceinline__ int share_of(int T, int W, int shares) {
    int i = (int)(__fdividef((float)T, (float)W) * (float)shares);
    while (share_begin(i, W, shares) > T) --i;
    while (share_begin(i + 1, W, shares) <= T) ++i;
    return i;
}

// Sum of a thread's number over the threads before it in its warp, and its own.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += n;
    }
    return v;
}

// Whether the places of all sequences are below 2^31. The host has seen to it for rows that
// are one sequence's each; where a start is below the one before it, they may be several's and
// their places many times as many, and what is counted in 32 bits would lead anywhere. All
// threads call it. (Rare; `total` is scratch.)
template <int G>
__device__ __noinline__ bool places_fit(const TreeArgs &a, unsigned long long *total) {
    if (threadIdx.x == 0) *total = 0;
    __syncthreads();
    unsigned long long mine = 0;
#pragma unroll 1
    for (int s = threadIdx.x; s < a.num_seqs; s += kThreads) mine += tree_seq_places(load_seq<G>(a, s), a.num_kv_heads);
    atomicAdd(total, mine);
    __syncthreads();
    return *static_cast<volatile unsigned long long *>(total) <= INT_MAX;
}

// The places of a lane, its shares, and this CTA's first piece (in `first`, shared memory);
// false when it has none. All threads call it; `sums` is scratch. A chain of dependent steps
// that every CTA goes through before its first tile: of up to kThreads sequences thread i
// has the i-th, which is scanned and summed at once, and there are no divisions but those
// that a batch needs: 4100 to 5800 cycles, of which 2000 wait for the lengths (with two
// scans and every division 1100 more).
template <int G>
__device__ __noinline__ bool plan_share(const TreeArgs &a, Walk *first, volatile int *sums, int &W, int &shares) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = a.num_seqs, Hkv = a.num_kv_heads;
    Seq mine{};
    int own = 0;                                // places of this thread's sequence of the first kThreads
    unsigned later = 0;                         // of those after them
    unsigned most = 0, least = INT_MAX;         // pairs of a sequence
    bool falls = false;                         // a start is below the one before it
#pragma unroll 1
    for (int s = tid; s < S; s += kThreads) {
        const Seq q = load_seq<G>(a, s);
        const int places = tree_seq_places(q, Hkv);
        falls |= q.n < 0;
        if (s == tid) {
            mine = q;
            own = places;
        } else {
            later += places;
        }
        if (q.pairs == 0) continue;
        most = max(most, q.pairs);
        least = min(least, q.pairs);
    }
    int scan = warp_scan(own, lane);
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (S > kThreads) later = __reduce_add_sync(0xffffffffu, later);
    if (lane == 31) {
        sums[warp] = scan;
        sums[32 + warp] = most;
        sums[64 + warp] = least;
        sums[96 + warp] = later;
    }
    if (tid == 0) first->T1 = -1;               // nothing found yet
    if (__syncthreads_or(falls) && !places_fit<G>(a, reinterpret_cast<unsigned long long *>(const_cast<int *>(sums + 128))))
        return false;
    // every warp adds up all warps' sums
    const bool there = lane < kWarpsAll;
    const int x = there ? sums[lane] : 0;
    most = __reduce_max_sync(0xffffffffu, there ? sums[32 + lane] : 0);
    least = __reduce_min_sync(0xffffffffu, there ? sums[64 + lane] : INT_MAX);
    int chunk = (int)__reduce_add_sync(0xffffffffu, (unsigned)x);
    int excl = scan - own + (int)__reduce_add_sync(0xffffffffu, (unsigned)(lane < warp ? x : 0));
    W = chunk;
    if (S > kThreads) W += (int)__reduce_add_sync(0xffffffffu, there ? (unsigned)sums[96 + lane] : 0u);
    // where all have the same number of pairs, the pairs are lanes
    const int lanes = tree_lanes((int)most, (int)least, a.workers);
    const bool side = lanes > 1;
    shares = a.workers;
    int w = blockIdx.x, my_lane = 0;
    if (side) {
        W /= lanes;
        shares /= lanes;
        w /= lanes;
        my_lane = blockIdx.x - w * lanes;
    }
    shares = max(1, min(W, shares));
    if (w >= shares || W == 0) return false;
    const int T0 = share_begin(w, W, shares), T1 = share_begin(w + 1, W, shares);
    int base = 0;
#pragma unroll 1
    for (int c0 = 0;;) {
        if (side) {
            own /= lanes;
            excl /= lanes;
            chunk /= lanes;
        }
        excl += base;
        if (own > 0 && T0 >= excl && T0 < excl + own) {
            const int rem = T0 - excl, places = mine.nt + kUnitPlaces;
            const int unit = rem / places;
            int kvh = unit, pair = 0;
            if (mine.pairs > lanes) {           // (not side by side)
                kvh = unit / mine.pairs;
                pair = unit - kvh * mine.pairs;
            }
            first->T = T0;
            first->T1 = T1;
            first->q = mine;
            first->s = c0 + tid;
            first->lane = my_lane;
            first->lanes = lanes;
            first->kvh = kvh;
            first->pair = my_lane + lanes * pair;
            first->j0 = rem - unit * places;
            if (first->j0 < mine.nt) piece_end(*first);
            else if (!next_unit<G>(*first, a)) first->T1 = -1;      // past the unit's tiles
        }
        base += chunk;
        c0 += kThreads;
        if (c0 >= S || base > T0) break;
        own = 0;
        if (c0 + tid < S) {
            mine = load_seq<G>(a, c0 + tid);
            own = tree_seq_places(mine, Hkv);
        }
        scan = warp_scan(own, lane);
        __syncthreads();                        // the sums before have been read
        if (lane == 31) sums[warp] = scan;
        __syncthreads();
        const int y = there ? sums[lane] : 0;
        chunk = (int)__reduce_add_sync(0xffffffffu, (unsigned)y);
        excl = scan - own + (int)__reduce_add_sync(0xffffffffu, (unsigned)(lane < warp ? y : 0));
    }
    __syncthreads();
    return first->T1 >= 0;
}

// -- masks -----------------------------------------------------------------------

// Of the 128 tokens from node b on (negative: before the first, in the context), those that
// a row of `words` mask words sees: all of the context, and the nodes below n whose bits it
// has.
__device__ __noinline__ uint4 seen_nodes(const uint32_t *row, int words, int b, int n) {
    uint32_t w[5], v[4];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        const int i = (b >> 5) + k;
        w[k] = i < 0 ? ~0u : (i < words ? row[i] : 0u);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int left = n - b - 32 * k;
        const uint32_t real = left <= 0 ? 0u : (left >= 32 ? ~0u : (1u << left) - 1u);
        v[k] = __funnelshift_r(w[k], w[k + 1], b & 31) & real;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Whether a piece's rows reach into query tile B. Its two streams are then the two query
// tiles over all key tiles; otherwise they are the even and the odd key tiles of query tile
// A (counted from the piece's first), merged when the piece ends.
template <int G>
__device__ __forceinline__ bool two_tiles(const volatile Walk &w) {
    return w.pair * (kPair / G) + kRows / G < w.q.n;
}
// Rows of a warp's 32 TMEM lanes: all, or the first 16 or 8 for up to 64 or 32 rows.
template <int G>
__device__ __forceinline__ int rows_per_warp(const volatile Walk &w) {
    const int tokens = w.q.n - w.pair * (kPair / G);
    return tokens <= 32 / G && G <= 8 ? 8 : (tokens <= 64 / G ? 16 : 32);
}
// Key tiles of a stream.
__device__ __forceinline__ int stream_tiles(int nt, bool two, int t) { return two ? nt : (nt + 1 - t) / 2; }

// 16-token groups of key tile j that hold keys.
__device__ __forceinline__ int groups_used(const volatile Walk &w, int j) {
    const int n = (w.q.L - j * kKeys + kGroup - 1) / kGroup;
    return n < 0 ? 0 : (n > kGroups ? kGroups : n);
}

// Whether key tile j reaches the nodes: its keys are masked, its V cleaned.
__device__ __forceinline__ bool reaches_nodes(const volatile Walk &w, int j) {
    return (j + 1) * kKeys > w.q.L - w.q.n;
}

// A V tile in shared memory whose keys reach the nodes: rows past the last token become
// zero, and so do the elements of nodes' rows that are not finite; the words of 32 nodes
// that had some are marked in `odd`. By the 128 threads of a stream. The 16-byte chunks of a
// row are permuted within it (128-byte swizzle), which does not matter here.
__device__ __noinline__ void clean_v(const volatile Walk &w, int j, uint8_t *vtile, uint32_t *odd, int words,
                                        int thread) {
    const int node0 = j * kKeys - (w.q.L - w.q.n);              // node of the tile's first key
    const int first = node0 < 0 ? -node0 : 0, left = w.q.L - j * kKeys;
    const int rows = groups_used(w, j) * kGroup - first;
    auto place = [&](int i) {
        return reinterpret_cast<uint4 *>(vtile + ((i >> 3) & 1) * kKVHalf + (first + (i >> 4)) * 128 + (i & 7) * 16);
    };
    constexpr int kBatch = 4;                                   // chunks a thread has in flight
#pragma unroll 1
    for (int i0 = thread; i0 < rows * 16; i0 += kRows * kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + kRows * k;
            const bool real = first + (i >> 4) < left;
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (i < rows * 16 && real) x[k] = *place(i);
            if (i < rows * 16 && !real) *place(i) = x[k];
        }
        // an exponent of all ones is an infinity or NaN: one more carries into the sign's place
        uint32_t found = 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            for (uint32_t v : {x[k].x, x[k].y, x[k].z, x[k].w}) found |= (v & 0x7f807f80u) + 0x00800080u;
        if (!(found & 0x80008000u)) continue;                   // as nearly all
#pragma unroll 1
        for (int i = i0; i < min(i0 + kRows * kBatch, min(left - first, rows) * 16); i += kRows) {
            uint4 v = *place(i);
            bool odd_one = false;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const bool lo = (v.x & 0x7f80u) == 0x7f80u, hi = (v.x & 0x7f800000u) == 0x7f800000u;
                odd_one |= lo || hi;
                v = make_uint4(v.y, v.z, v.w, v.x & (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u));
            }
            *place(i) = v;
            const int node = node0 + first + (i >> 4);
            if (odd_one && node < 32 * words) atomicOr(odd, 1u << (node >> 5));     // the others nobody sees
        }
    }
}

// What clean_v took out of the nodes that a row sees among tokens [t0, t1), added to its
// written result: dims [d0, d1) of those that are not finite. `out` is the row in bf16, or
// `part` its words of a part in fp32. Rare.
__device__ __noinline__ void add_odd(const TreeArgs &a, uint32_t odd, int s, int kvh, int first_node, int t0, int t1,
                                     const uint32_t *mask_row, uint16_t *out, float4 *part, int d0, int d1) {
    const int lb = a.block_size_log2;
    for (; odd; odd &= odd - 1) {
        const int i = __ffs(odd) - 1;
        for (uint32_t bits = mask_row[i]; bits; bits &= bits - 1) {
            const int t = first_node + 32 * i + __ffs(bits) - 1;
            if (t < t0 || t >= t1) continue;
            const int64_t bid = __ldg(a.block_tables + (int64_t)s * a.max_blocks_per_seq + (t >> lb));
            const int off = t & ((1 << lb) - 1);
            if (bid < 0 || bid >= a.num_blocks) continue;       // read as zeros
            const int64_t row = a.head_major ? ((bid * a.num_kv_heads + kvh) << lb) + off
                                             : ((bid << lb) + off) * a.num_kv_heads + kvh;
            const uint16_t *v = static_cast<const uint16_t *>(a.v_cache) + row * kHeadDim;
            for (int d = d0; d < d1; ++d) {
                if ((v[d] & 0x7f80) != 0x7f80) continue;
                const float x = __uint_as_float((uint32_t)v[d] << 16);
                if (out) {
                    const float y = __uint_as_float((uint32_t)out[d] << 16) + x;
                    out[d] = (uint16_t)(pack_bf16x2(y, y) & 0xffffu);
                } else {
                    reinterpret_cast<float *>(part + (d >> 2) * kPair)[d & 3] += x;
                }
            }
        }
    }
}

// Rows of a TMA box of queries: whole tokens' G heads, and whole 8-row swizzle atoms.
__host__ __device__ constexpr int box_rows(int G) { return G > 8 ? G : 8; }

// The two buffers of queries, counted alike by the V warp, which fills them, and the MMA
// warp: a piece of two query tiles takes both, others take them in turn.
struct QBuffers {
    int n0 = 0, n1 = 0, next = 0;
    // the buffer of query tile A
    __device__ __forceinline__ int take(bool two) {
        const int b = two ? 0 : next;
        if (!two) next ^= 1;
        n0 += two || b == 0 ? 1 : 0;
        n1 += two || b == 1 ? 1 : 0;
        return b;
    }
    __device__ __forceinline__ int uses(int b) const { return b == 0 ? n0 : n1; }
    // one that was taken and not filled
    __device__ __forceinline__ void drop(int b) {
        if (b == 0) --n0;
        else --n1;
    }
};

// -- softmax of one key tile ----------------------------------------------------------
//
// Scores S from TMEM (of -Q, where the scale is negative, so that sc is positive), the masked
// ones -infinity; the running max m (log2 units) is raised
// only when the tile exceeds it by 2^8: weights stay below 2^8, far inside fp32 and bf16
// range, and O is rescaled rarely. P = 2^(S sc - m), rounded to bf16 for the second product,
// whose operands have to be: its error of up to 2^-8 of a weight averages out over the keys
// (0.0019 to 0.0024 of a result's length against 64 bits, where rounding the result itself is
// 0.0017). The sum is of the exact weights.

// The new max for a tile whose largest raw score is `most` (-infinity: all masked); the
// factor on what was summed before (1 when the max stays).
__device__ __forceinline__ float raise_max(float most, float sc, float &m, float &lsum) {
    const float mt = most * sc;
    if (!(mt > m + kRescaleSlack)) return 1.f;
    const float alpha = m != -INFINITY ? ex2(m - mt) : 1.f;
    lsum *= alpha;
    m = mt;
    return alpha;
}

// A tile of whose scores none passes a row's reference by more than the slack, as nearly all
// do once a few tiles have set it: the weights against the reference as it is, and the
// maximum beside them, in one reading. False, with nothing changed, when a row of the warp
// has to raise it.
__device__ __forceinline__ bool steady_tile(uint32_t tS, float sc, float m, float &lsum) {
    if (__any_sync(0xffffffffu, m == -INFINITY)) return false;
    float e[2] = {-INFINITY, -INFINITY};
    uint32_t sr[2][32], pw[2][32];
    const Two sc2{sc, sc}, mb2{-m, -m};
    Two l2[2] = {};
    tc::tmem_ld32(tS, sr[0]);
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
        tc::tmem_ld_wait();
        if (ch < 3) tc::tmem_ld32(tS + 32 * (ch + 1), sr[(ch + 1) & 1]);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const Two s2{__uint_as_float(sr[ch & 1][2 * c]), __uint_as_float(sr[ch & 1][2 * c + 1])};
            const Two x = fma2(s2, sc2, mb2);
            const Two p{ex2(x.x), ex2(x.y)};
            e[c & 1] = fmax3(e[c & 1], s2.x, s2.y);
            l2[c & 1] = add(l2[c & 1], p);
            pw[ch >> 1][16 * (ch & 1) + c] = pack_bf16x2(p.x, p.y);
        }
    }
    if (__any_sync(0xffffffffu, fmaxf(e[0], e[1]) * sc > m + kRescaleSlack)) return false;
    tc::tmem_st32(tS, pw[0]);
    tc::tmem_st32(tS + 32, pw[1]);
    lsum += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
    tc::tmem_st_wait();
    return true;
}

// A thread per row: 128 scores of its TMEM lane, 32 at a time, once for the maximum and
// again for the weights: held all at once they take four times the code.
__device__ __forceinline__ void wide_tile(uint32_t tS, uint32_t tO, float sc, bool nodes,
                                          const uint32_t (&vis)[4], float &m, float &lsum) {
    float e[2] = {-INFINITY, -INFINITY};
    uint32_t sr[2][32];
    tc::tmem_ld32(tS, sr[0]);
    if (nodes) {
        uint32_t v0 = vis[0], v1 = vis[1], v2 = vis[2], v3 = vis[3];
#pragma unroll 1
        for (int ch = 0; ch < 4; ch += 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                tc::tmem_ld_wait();
                if (ch + h < 3) tc::tmem_ld32(tS + 32 * (ch + h + 1), sr[h ^ 1]);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    if (!(v0 >> c & 1)) sr[h][c] = kMasked;
                    e[c & 1] = fmaxf(e[c & 1], __uint_as_float(sr[h][c]));
                }
                tc::tmem_st32(tS + 32 * (ch + h), sr[h]);
                v0 = v1;
                v1 = v2;
                v2 = v3;
            }
        }
        tc::tmem_st_wait();
    } else {
#pragma unroll 1
        for (int ch = 0; ch < 4; ch += 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                tc::tmem_ld_wait();
                if (ch + h < 3) tc::tmem_ld32(tS + 32 * (ch + h + 1), sr[h ^ 1]);
#pragma unroll
                for (int c = 0; c < 32; c += 4)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        e[k] = fmax3(e[k], __uint_as_float(sr[h][c + 2 * k]), __uint_as_float(sr[h][c + 2 * k + 1]));
            }
        }
    }
    tc::tmem_ld32(tS, sr[0]);
    const float alpha = raise_max(fmaxf(e[0], e[1]), sc, m, lsum);
    const float mb = m == -INFINITY ? 0.f : m;
    const Two sc2{sc, sc}, mb2{-mb, -mb};
    Two l2[2] = {};
#pragma unroll 1
    for (int ch = 0; ch < 4; ch += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            tc::tmem_ld_wait();
            if (ch + h < 3) tc::tmem_ld32(tS + 32 * (ch + h + 1), sr[h ^ 1]);
            uint32_t pw[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const Two x = fma2(Two{__uint_as_float(sr[h][2 * c]), __uint_as_float(sr[h][2 * c + 1])}, sc2, mb2);
                const Two p{ex2(x.x), ex2(x.y)};
                l2[c & 1] = add(l2[c & 1], p);
                pw[c] = pack_bf16x2(p.x, p.y);
            }
            // over columns that have been read
            tc::tmem_st16(tS + (ch + h) * 16, pw);
        }
    }
    lsum += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
    if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
            uint32_t o[32];
            tc::tmem_ld32(tO + ch * 32, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tc::tmem_st32(tO + ch * 32, o);
        }
    }
    tc::tmem_st_wait();
}

// A quad of lanes per row, or (R = 2) per row and the one 8 further on: lane q of a quad
// has scores 8 k + 2 q and the next, k = 0 .. 15, of each.
template <int R>
__device__ __forceinline__ void narrow_tile(uint32_t tS, uint32_t tO, float sc, bool nodes,
                                            const uint32_t (&vis)[R][4], float (&m)[R], float (&lsum)[R]) {
    const int q2 = 2 * (threadIdx.x & 3);
    uint32_t s[64];
    tc::tmem_ld_16x256b_x16(tS, s);
    tc::tmem_ld_wait();
    float alpha[2] = {1.f, 1.f}, mb[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < R; ++x) {
        if (nodes) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint32_t v = vis[x][k >> 2] >> q2;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (!(v >> (8 * (k & 3) + e) & 1)) s[4 * k + 2 * x + e] = kMasked;
            }
        }
        float e2[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 16; ++k)
            e2[k & 1] = fmax3(e2[k & 1], __uint_as_float(s[4 * k + 2 * x]), __uint_as_float(s[4 * k + 2 * x + 1]));
        float most = fmaxf(e2[0], e2[1]);
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        alpha[x] = raise_max(most, sc, m[x], lsum[x]);
        mb[x] = m[x] == -INFINITY ? 0.f : m[x];
    }
    uint32_t pw[32];
    float l2[2][2] = {};
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (x >= R) {                       // no row there
                pw[2 * k + x] = 0u;
                continue;
            }
            const float p0 = ex2(fmaf(__uint_as_float(s[4 * k + 2 * x]), sc, -mb[x]));
            const float p1 = ex2(fmaf(__uint_as_float(s[4 * k + 2 * x + 1]), sc, -mb[x]));
            l2[x][k & 1] += p0 + p1;
            pw[2 * k + x] = pack_bf16x2(p0, p1);
        }
    tc::tmem_st_16x128b_x16(tS, pw);
#pragma unroll
    for (int x = 0; x < R; ++x) lsum[x] += l2[x][0] + l2[x][1];
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            tc::tmem_ld_16x256b_x8(tO + 64 * h, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[(i >> 1) & 1]);
            tc::tmem_st_16x256b_x8(tO + 64 * h, o);
        }
    }
    tc::tmem_st_wait();
}

// An element of a result from those of both streams; a row that saw nothing outputs zero,
// whatever its O. (A second O that is not there may be anything.)
__device__ __forceinline__ float merged(uint32_t o, uint32_t o2, float fa, bool b_too, float fb, bool none) {
    const float x = __uint_as_float(o) * fa, y = fmaf(__uint_as_float(o2), fb, x);
    return none ? 0.f : (b_too ? y : x);
}
__device__ __forceinline__ uint4 pack(const float *f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Lane i of a quad gives its 16 bytes k to lane k, as that one's i-th: a store of 32 lanes then
// covers 64 bytes of 8 rows instead of 16 of 32.
__device__ __forceinline__ void quad_transpose(uint4 (&x)[4], int lane) {
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & m) continue;
            uint4 &lo = x[k], &hi = x[k | m];
            uint4 v = up ? lo : hi;
            v.x = __shfl_xor_sync(0xffffffffu, v.x, m);
            v.y = __shfl_xor_sync(0xffffffffu, v.y, m);
            v.z = __shfl_xor_sync(0xffffffffu, v.z, m);
            v.w = __shfl_xor_sync(0xffffffffu, v.w, m);
            if (up) lo = v;
            else hi = v;
        }
    }
}

// What a softmax warp counts over its pieces.
struct Streams {
    uint32_t gt = 0, ga = 0;    // key tiles before this piece, of this stream and of all
    int piece = 0, halves = 0;  // pieces before this one; those whose streams were halves
};

// A softmax warp's part of one piece: R = 0 a thread per row, 1 and 2 a quad of lanes per one
// and two rows. False when a wait ran out.
template <int G, int R>
__device__ __forceinline__ bool softmax_piece(const TreeArgs &a, const volatile Walk &w, Streams &st, uint8_t *smem,
                                              uint32_t sbase, uint32_t tmem) {
    constexpr int NR = R == 2 ? 2 : 1;                  // rows of a thread
    const int tid = threadIdx.x, wg = tid >> 7, r = tid & 127;
    const uint32_t lane = (uint32_t)(r & ~31) << 16;
    const uint32_t tS = tmem + lane + wg * 256, tO = tS + 128;
    auto bar = [&](uint32_t i) { return sbase + kOffCtl + 8 * i; };
    volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffAbort);
    uint32_t *odd_marks = reinterpret_cast<uint32_t *>(smem + kOffOdd);
    const float sc = fabsf(a.scale_log2);
    const bool two = R == 0 && two_tiles<G>(w);
    const int nt = w.j1 - w.j0, ntt = stream_tiles(nt, two, wg);
    const int tile = two ? wg : 0;                      // query tile
    // this thread's first row of the query tile, the other is 8 further on
    const int row0 = R == 0 ? r : (r >> 5) * (8 * R) + ((tid >> 2) & 7);
    auto token = [&](int row) { return w.pair * (kPair / G) + tile * (kRows / G) + row / G; };
    auto row_valid = [&](int row) { return token(row) < w.q.n && row % G < a.group; };
    bool rv[NR];
#pragma unroll
    for (int x = 0; x < NR; ++x) rv[x] = row_valid(row0 + 8 * x);
    // warps past the last row only take part in the hand-offs and the cleaning
    const bool any = __any_sync(0xffffffffu, rv[0]);
    float m[NR], lsum[NR];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
        m[x] = -INFINITY;
        lsum[x] = 0.f;
    }
#pragma unroll 1
    for (int j = 0; j < ntt; ++j) {
        const int jj = two ? j : 2 * j + wg;            // key tile, from the piece's first
        const int b0 = (w.j0 + jj) * kKeys - (w.q.L - w.q.n);       // node of its first key
        const bool nodes = b0 + kKeys > 0;
        uint32_t vis[NR][4];
        if (nodes && any)
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                const uint32_t *row = a.mask + ((int64_t)w.q.q0 + token(row0 + 8 * x)) * a.mask_words;
                const uint4 v = rv[x] ? seen_nodes(row, a.mask_words, b0, w.q.n) : make_uint4(0u, 0u, 0u, 0u);
                vis[x][0] = v.x;
                vis[x][1] = v.y;
                vis[x][2] = v.z;
                vis[x][3] = v.w;
            }
        // S_t(j) done: also PV_t(j - 1), issued before it, so O is stable (a warp without
        // rows sleeps until then: its polls would take from the others)
        if (!warp_wait(bar(kBarSFull + wg), (st.gt + j) & 1, abort, any)) return false;
        tc::fence_after_sync();
        if (any) {
            if constexpr (R == 0) {
                if (nodes || !steady_tile(tS, sc, m[0], lsum[0])) wide_tile(tS, tO, sc, nodes, vis[0], m[0], lsum[0]);
            } else narrow_tile<R>(tS, tO, sc, nodes, vis, m, lsum);
        }
        // V has to be there to be cleaned; of two query tiles A's warps do it, whose product
        // is issued first
        if (nodes && (!two || wg == 0)) {
            const uint32_t g = st.ga + jj;
            if (!warp_wait(bar(kBarVFull + g % kVStages), (g / kVStages) & 1, abort, any)) return false;
            clean_v(w, w.j0 + jj, smem + kOffV + (g % kVStages) * kKVBytes, odd_marks + st.piece % kOddSets, a.mask_words, r);
            tc::fence_proxy_async();
        }
        tc::fence_before_sync();
        warp_arrive(bar(kBarPReady + wg));
    }
    if (ntt > 0) {
        if (!warp_wait(bar(kBarPVDone + wg), (st.gt + ntt - 1) & 1, abort, any)) return false;
        tc::fence_after_sync();
    }
    if (R > 0) {
        // a quad's sums; its maxima are common
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            lsum[x] += __shfl_xor_sync(0xffffffffu, lsum[x], 1);
            lsum[x] += __shfl_xor_sync(0xffffffffu, lsum[x], 2);
        }
    }
    // Streams that are halves of the same rows: both know both maxima and sums, stream A
    // takes dims 0-63 of both O, stream B the others (both warps of a row have its TMEM lane).
    const bool first = R == 0 || (tid & 3) == 0;        // of the row's lanes
    float fa[NR], fb[NR];                               // factors on the O of A, B (own: fa)
#pragma unroll
    for (int x = 0; x < NR; ++x) {
        fa[x] = 1.f;
        fb[x] = 0.f;
    }
    if (!two) {
        // (a stream without tiles has not waited for the last piece's to be read)
        if (ntt == 0 && st.piece > 0 && !warp_wait(bar(kBarOFree), (st.piece - 1) & 1, abort)) return false;
        float2 *ml = reinterpret_cast<float2 *>(smem + kOffHalves);
#pragma unroll
        for (int x = 0; x < NR; ++x)
            if (first) ml[wg * kRows + row0 + 8 * x] = make_float2(m[x], lsum[x]);
        tc::fence_before_sync();
        warp_arrive(bar(kBarHalves));
        if (!warp_wait(bar(kBarHalves), st.halves & 1, abort, any)) return false;
        tc::fence_after_sync();
        ++st.halves;
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const float2 ea = ml[row0 + 8 * x], eb = ml[kRows + row0 + 8 * x];
            m[x] = fmaxf(ea.x, eb.x);
            fa[x] = ea.y == 0.f ? 0.f : ex2(ea.x - m[x]);
            fb[x] = eb.y == 0.f ? 0.f : ex2(eb.x - m[x]);
            lsum[x] = (ea.y == 0.f ? 0.f : ea.y * fa[x]) + (eb.y == 0.f ? 0.f : eb.y * fb[x]);
        }
    }
    if (any) {
        const bool whole = w.j0 == 0 && w.j1 == w.q.nt, b_too = !two && nt > 1;
        // a row's place in the output (16-byte words), and among the parts
        auto out_row = [&](int row) {
            return reinterpret_cast<uint4 *>(a.out) +
                   (((int64_t)w.q.q0 + token(row)) * a.num_q_heads + (int64_t)w.kvh * a.group + row % G) * (kHeadDim / 8);
        };
        const int slot = 2 * (int)blockIdx.x + (w.j0 == 0 ? 1 : 0);
        float4 *po = a.part_o + (int64_t)slot * 32 * kPair + tile * kRows;
        const int d0 = two ? 0 : 64 * wg, d1 = two ? kHeadDim : d0 + 64;
        bool none[NR];
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const float inv = whole ? 1.f / lsum[x] : 1.f;
            none[x] = lsum[x] == 0.f;
            fa[x] *= inv;
            fb[x] *= inv;
            if (!whole && rv[x] && first && (two || wg == 0))
                a.part_ml[(int64_t)slot * kPair + tile * kRows + row0 + 8 * x] = make_float2(m[x], lsum[x]);
        }
        if constexpr (R == 0) {
            if (two) {
                // the rows of a quad of lanes are written together
                uint4 *const quad = out_row(row0 & ~3) + (tid & 3);
                const unsigned valid = __ballot_sync(0xffffffffu, rv[0]) >> (tid & 28);
#pragma unroll 1
                for (int d = 0; d < kHeadDim; d += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32(tO + d, o);
                    tc::tmem_ld_wait();
                    float y[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) y[c] = none[0] ? 0.f : __uint_as_float(o[c]) * fa[0];
                    if (whole) {
                        uint4 x[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) x[c] = pack(y + 8 * c);
                        quad_transpose(x, tid);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (valid >> k & 1) quad[(k / G * a.num_q_heads + k % G) * (kHeadDim / 8) + d / 8] = x[k];
                    } else if (rv[0]) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            po[((d + c) / 4) * kPair + row0] = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
                    }
                }
            } else {
                uint4 *const orow = out_row(row0);
#pragma unroll 1
                for (int d = d0; d < d1; d += 16) {
                    uint32_t o[16], o2[16];
                    tc::tmem_ld16(tmem + lane + 128 + d, o);
                    tc::tmem_ld16(tmem + lane + 384 + d, o2);
                    tc::tmem_ld_wait();
                    float y[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) y[c] = merged(o[c], o2[c], fa[0], b_too, fb[0], none[0]);
#pragma unroll
                    for (int c = 0; c < 16; c += 8) {
                        if (rv[0] && whole) {
                            orow[(d + c) / 8] = pack(y + c);
                        } else if (rv[0]) {
                            po[((d + c) / 4) * kPair + row0] = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
                            po[((d + c) / 4 + 1) * kPair + row0] = make_float4(y[c + 4], y[c + 5], y[c + 6], y[c + 7]);
                        }
                    }
                }
            }
        } else {
            // (halves) dims d + 2 (lane % 4) and the next
            uint32_t *orow[NR];
            float2 *prow[NR];
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                const int pairs = (tid & 3) + d0 / 2;
                orow[x] = reinterpret_cast<uint32_t *>(out_row(row0 + 8 * x)) + pairs;
                prow[x] = reinterpret_cast<float2 *>(po + (pairs >> 1) * kPair + row0 + 8 * x) + (pairs & 1);
            }
#pragma unroll 1
            for (int d = 0; d < 64; d += 32) {
                uint32_t o[16], o2[16];
                tc::tmem_ld_16x256b_x4(tmem + lane + 128 + d0 + d, o);
                tc::tmem_ld_16x256b_x4(tmem + lane + 384 + d0 + d, o2);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int x = 0; x < NR; ++x) {
                        const int i = 4 * k + 2 * x;
                        const float y0 = merged(o[i], o2[i], fa[x], b_too, fb[x], none[x]);
                        const float y1 = merged(o[i + 1], o2[i + 1], fa[x], b_too, fb[x], none[x]);
                        if (rv[x] && whole) orow[x][(d + 8 * k) / 2] = pack_bf16x2(y0, y1);
                        else if (rv[x]) prow[x][(d + 8 * k) / 2 * kPair] = make_float2(y0, y1);
                    }
            }
        }
        const uint32_t odd = reaches_nodes(w, w.j1 - 1)
            ? reinterpret_cast<volatile uint32_t *>(odd_marks)[st.piece % kOddSets] : 0u;
        if (odd) {
            __syncwarp();               // the row's lanes have written
#pragma unroll 1
            for (int x = 0; x < NR; ++x) {
                const int row = row0 + 8 * x;
                if (!first || !row_valid(row)) continue;
                add_odd(a, odd, w.s, w.kvh, w.q.L - w.q.n, w.j0 * kKeys, min(w.j1 * kKeys, w.q.L),
                        a.mask + ((int64_t)w.q.q0 + token(row)) * a.mask_words,
                        whole ? reinterpret_cast<uint16_t *>(out_row(row)) : nullptr, po + row, d0, d1);
            }
        }
    }
    // the marks of the piece after the next: everybody has read those of the piece before the
    // last, and nobody is there yet
    if (tid == 0) reinterpret_cast<volatile uint32_t *>(odd_marks)[(st.piece + 2) % kOddSets] = 0u;
    tc::fence_before_sync();
    warp_arrive(bar(kBarOFree));
    st.gt += ntt;
    st.ga += nt;
    ++st.piece;
    return true;
}

// -- attention ---------------------------------------------------------------------

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
tree_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap tmap_k,
            const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_q) {
    constexpr int BT = kRows / G;               // tokens per query tile
    constexpr int BR = box_rows(G);
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        tc::prefetch_map(&tmap_k);
        tc::prefetch_map(&tmap_v);
        tc::prefetch_map(&tmap_q);
    }
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {                        // the swizzle atoms need 1024-byte alignment
        if (tid == 0) set_error(kErrSmemAlign);
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        if (tid == 0) a.tasks[blockIdx.x] = make_int4(-1, 0, 0, 0);
        return;
    }
    const uint32_t ctl = sbase + kOffCtl;
    auto bar = [&](uint32_t i) { return ctl + 8 * i; };
    volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffAbort);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(kBarQFull + i), 1);
            tc::mbar_init(bar(kBarQEmpty + i), 1);
        }
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
        }
        tc::mbar_init(bar(kBarOFree), kSoftmaxThreads / 32);
        tc::mbar_init(bar(kBarHalves), kSoftmaxThreads / 32);
        tc::mbar_init(bar(kBarDrain), 1);
        *abort = 0;
        for (int i = 0; i < kOddSets; ++i) reinterpret_cast<uint32_t *>(smem + kOffOdd)[i] = 0u;
        tc::fence_mbar_init();
    }
    if (warp == kMmaWarp) tc::tmem_alloc(sbase + kOffTmemSlot, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffTmemSlot);

    // programmatic dependent of whatever precedes the call
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    int W, shares;
    Walk *walks = reinterpret_cast<Walk *>(smem + kOffWalk);
    const bool works = plan_share<G>(a, walks + kWarpsAll, reinterpret_cast<volatile int *>(smem + kOffHalves), W, shares);
    // the place of the first piece, for each warp its own
    if ((tid & 31) < kWalkBytes / 4)
        reinterpret_cast<volatile int *>(walks + warp)[tid & 31] =
            reinterpret_cast<volatile int *>(walks + kWarpsAll)[tid & 31];
    __syncwarp();
    volatile Walk &w = walks[warp];
    const int w_id = blockIdx.x;
    if (warp == kVWarp && (tid & 31) == 0) a.tasks[w_id] = make_int4(-1, 0, 0, 0);
    if (!works) {
        // more CTAs than shares, or a share of no tiles
    } else if (tid < kSoftmaxThreads) {
        // ---------------- softmax warpgroups ----------------
        Streams st;
        bool ok = true;
#pragma unroll 1
        do {
            switch (rows_per_warp<G>(w)) {
                case 8: ok = softmax_piece<G, 1>(a, w, st, smem, sbase, tmem); break;
                case 16: ok = softmax_piece<G, 2>(a, w, st, smem, sbase, tmem); break;
                default: ok = softmax_piece<G, 0>(a, w, st, smem, sbase, tmem);
            }
        } while (ok && walk_next<G>(w, a));
    } else if (warp == kKWarp || warp == kVWarp) {
        // ---------------- K and V producers ----------------
        const bool is_v = warp == kVWarp;
        const int nst = is_v ? kVStages : kKStages;
        const int lane = tid & 31;
        const int q = lane >> 1, h = lane & 1;      // this lane's box of a tile, and its half of the dims
        const uint32_t bar_full = bar(is_v ? kBarVFull : kBarKFull);
        const uint32_t bar_empty = bar(is_v ? kBarVEmpty : kBarKEmpty);
        const uint32_t base = sbase + (is_v ? kOffV : kOffK);
        const void *map = is_v ? static_cast<const void *>(&tmap_v) : static_cast<const void *>(&tmap_k);
        const int box = a.box_tokens, boxes = kKeys / box;
        uint32_t gt = 0;                            // tiles issued
        QBuffers qb;
        bool ok = true;
#pragma unroll 1
        do {
            if (is_v) {
                // the queries, once the products of the piece that had the buffer are done
                const bool two = two_tiles<G>(w);
                const int b0 = qb.take(two);
                for (int t = 0; t <= (two ? 1 : 0) && ok; ++t) {
                    const int b = b0 + t;
                    if (qb.uses(b) > 1) ok = warp_wait(bar(kBarQEmpty + b), qb.uses(b) & 1, abort);
                    if (!ok) {
                        qb.drop(b);
                        break;
                    }
                    // box q: rows BR q .. of the tile, in the first rq rows of every 32
                    const int rq = rows_per_warp<G>(w), nq = 4 * rq / BR;
                    if (lane == 0) tc::mbar_expect_tx(bar(kBarQFull + b), (uint32_t)(nq * 2 * BR * 128));
                    __syncwarp();
                    if (q < nq)
                        tc::tma_load_3d(sbase + kOffQ + b * kQBytes + h * kQHalf +
                                            (BR * q / rq * 32 + BR * q % rq) * 128,
                                        &tmap_q, h * 64, w.kvh * a.group,
                                        w.q.q0 + w.pair * 2 * BT + t * BT + BR * q / G, bar(kBarQFull + b));
                    warp_arrive(bar(kBarQFull + b));
                }
                if (!ok) break;
                // a unit that begins here and ends in another share: the combine's task
                if (lane == 0 && w.j0 == 0 && w.j1 < w.q.nt) {
                    const int parts = share_of(w.T + w.q.nt - 1, W, shares) - w_id / w.lanes + 1;
                    const int tokens = min(w.q.n - w.pair * (kPair / G), kPair / G);
                    a.tasks[w_id] = make_int4(w.q.q0 + w.pair * (kPair / G), w.kvh, tokens, parts | w.lanes << 8);
                }
                __syncwarp();
            }
            // coordinates (dim 1, dim 2) of this lane's box of tile j; dim 1 (or 2) at
            // -kKeys reads zeros, for a block id outside the pool; x = INT_MIN: no box. A box
            // may reach past the last token, but not past its block: those keys are masked,
            // their V rows cleaned.
            auto box_at = [&](int j) -> int2 {
                const int t = j * kKeys + q * box;
                if (q >= boxes || j >= w.j1 || t >= w.q.L) return make_int2(INT_MIN, 0);
                const int lb = a.block_size_log2;
                const int bid = __ldg(a.block_tables + (int64_t)w.s * a.max_blocks_per_seq + (t >> lb));
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
                if (!warp_wait(bar_empty + 8 * st, ((gt / nst) & 1) ^ 1, abort, true)) { ok = false; break; }
                const uint32_t full = bar_full + 8 * st;
                const int n = __popc(__ballot_sync(0xffffffffu, at.x != INT_MIN));
                if (lane == 0) tc::mbar_expect_tx(full, (uint32_t)(n * box * 128));
                __syncwarp();
                if (at.x != INT_MIN)
                    tc::tma_load_3d(base + st * kKVBytes + h * kKVHalf + q * box * 128, map, h * 64, at.x, at.y, full);
                // the test hook holds back one V arrival (set_prefill_fault)
                if (!(is_v && a.fault_hold_v && gt == 0)) warp_arrive(full);
                ++gt;
            }
        } while (ok && walk_next<G>(w, a));
        // the last fill of every stage, and the last queries, have landed
#pragma unroll 1
        for (uint32_t g = gt > (uint32_t)nst ? gt - nst : 0; g < gt; ++g)
            drain(bar_full + 8 * (g % nst), (g / nst) & 1);
#pragma unroll 1
        for (int b = 0; b < 2; ++b)
            if (qb.uses(b) > 0) drain(bar(kBarQFull + b), (qb.uses(b) - 1) & 1);
    } else if (warp == kMmaWarp) {
        // ---------------- MMA issue ----------------
        const uint64_t dq = tc::sw128_desc(sbase + kOffQ, 16, 1024);        // K-major
        const uint64_t dk = tc::sw128_desc(sbase + kOffK, 16, 1024);
        const uint64_t dv = tc::sw128_desc(sbase + kOffV, kKVHalf, 1024);   // MN-major: next 64 dims
        const uint32_t hi = (uint32_t)(dq >> 32);                           // same for all three
        const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
        auto desc = [hi](uint32_t lo) { return ((uint64_t)hi << 32) | lo; };
        const uint32_t idesc_s = kIdescS | (a.scale_log2 < 0.f ? kNegateA : 0u);
        // S of stream t from query buffer b and K stage st
        auto issue_s = [&](int t, int b, int st, uint32_t release) {
            const uint32_t qd = q_lo + b * (kQBytes >> 4);
            const uint32_t kd = k_lo + st * (kKVBytes >> 4);
            const uint32_t d = tmem + t * 256;
#pragma unroll
            for (int kk = 0; kk < kHeadDim / 16; ++kk)
                tc::mma_ss(d, desc(qd + (((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4)),
                           desc(kd + (((kk >> 2) * kKVHalf + (kk & 3) * 32) >> 4)), idesc_s, kk > 0);
            tc::commit(bar(kBarSFull + t));
            if (release) tc::commit(release);
        };
        // over the first nv 16-key groups (the rest have P = 0 and no V)
        auto issue_pv = [&](int t, int st, bool acc, int nv, uint32_t release) {
            const uint32_t vd = v_lo + st * (kKVBytes >> 4);
            const uint32_t pa_ = tmem + t * 256;
            const uint32_t d = pa_ + 128;
            tc::mma_ts(d, pa_, desc(vd), kIdescPV, acc);
            if (nv == kGroups) {
#pragma unroll
                for (int kk = 1; kk < kGroups; ++kk)
                    tc::mma_ts(d, pa_ + kk * 8, desc(vd + ((kk * 2048) >> 4)), kIdescPV, true);
            } else {
#pragma unroll 1
                for (int kk = 1; kk < nv; ++kk)
                    tc::mma_ts(d, pa_ + kk * 8, desc(vd + ((kk * 2048) >> 4)), kIdescPV, true);
            }
            tc::commit(bar(kBarPVDone + t));
            if (release) tc::commit(release);
        };
        auto await = [&](uint32_t b, uint32_t parity) { return lane_wait(b, parity, abort); };
        static_assert(kVStages == 2, "V stages are counted on in turn");
        // Step i is of stream i % 2: of two query tiles over key tile i / 2, of halves over key
        // tile i. In turn: PV of step i once its P is in TMEM (and, for the first of a piece,
        // the previous piece's results have been read), then S of step i + 2. The tiles they
        // need have been waited for before, off the chain from P to S. A stage is released
        // after its last reader.
        // (One lane does all of it: an elected lane a product had the warp part and meet four
        // times a step, 304 us against 298. A wait costs 50 to 100 cycles also where nothing is to
        // wait for: a second reader does not wait for its tiles, and the rings' places are
        // counted on. Tiles seen by a softmax warp, so that P alone is waited for here, made it
        // 289 against 277: what looks like waiting for V is the queue of products.)
        int vs = 0, ks = 0;                     // next V and K stage, and their phases
        uint32_t v_phase = 0, k_phase = 0, p_phase = 0;         // (p_phase: bit t, of stream t)
        int piece = 0;
        QBuffers qb;
        bool ok = true;
#pragma unroll 1
        do {
            const int nt = w.j1 - w.j0;
            const bool two = two_tiles<G>(w);
            const int steps = nt << (two ? 1 : 0);
            const int tail = groups_used(w, w.j1 - 1);          // 16-key groups of the last tile
            const int b0 = qb.take(two);
            if (tc::elect_one()) {
                ok = await(bar(kBarQFull + b0), (qb.uses(b0) - 1) & 1);
                if (ok && two) ok = await(bar(kBarQFull + 1), (qb.uses(1) - 1) & 1);
#pragma unroll 1
                for (int i = -2; ok && i < steps; ++i) {
                    const int t = i & 1;
                    const bool first = !two || t == 0, last = !two || t == 1;       // reader of its tiles
                    const bool more = i + 2 < steps;
                    if (first) {
                        if (i >= 0) ok = await(bar(kBarVFull + vs), v_phase);
                        if (ok && more) ok = await(bar(kBarKFull + ks), k_phase);
                        if (ok && i == 0 && piece > 0) ok = await(bar(kBarOFree), (piece - 1) & 1);
                    }
                    if (ok && i >= 0) ok = await(bar(kBarPReady + t), p_phase >> t & 1);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (i >= 0) {
                        issue_pv(t, vs, i > 1, i + (two ? 2 : 1) < steps ? kGroups : tail, last ? bar(kBarVEmpty + vs) : 0u);
                        p_phase ^= 1u << t;
                        if (last) {
                            vs ^= 1;
                            v_phase ^= vs == 0 ? 1u : 0u;
                        }
                    }
                    if (more) {
                        issue_s(t, two ? t : b0, ks, last ? bar(kBarKEmpty + ks) : 0u);
                        if (last) {
                            ks = ks == kKStages - 1 ? 0 : ks + 1;
                            k_phase ^= ks == 0 ? 1u : 0u;
                        }
                        // the queries' buffers are free once the piece's last scores are there
                        if (i + 3 == steps) {
                            tc::commit(bar(kBarQEmpty + b0));
                            if (two) tc::commit(bar(kBarQEmpty + 1));
                        }
                    }
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            ++piece;
        } while (ok && walk_next<G>(w, a));
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

// Merge of the parts of the units that one worker began and others ended, 8 rows x 32 words
// of 4 dims at a time. A part's words are [dim / 4][row]. Every CTA counts the groups of 8
// rows of all such units and takes every gridDim.x-th: few units of many parts then have as
// many CTAs as many of few. (A CTA for each group that there could be, 32 a worker, takes
// 4 us where no unit has parts; 4 a worker for its own unit's alone take 15 us more for 10
// units of 15 parts.)
constexpr int kCombineCtas = 4;              // per worker
constexpr int kCombineBatch = 4;             // parts whose loads are in flight together
constexpr int kCombineThreads = kCombineRows * 32;
static_assert(kTreeMaxWorkers <= kCombineThreads, "a thread for each worker");

template <int G>
__global__ void __launch_bounds__(kCombineThreads) tree_combine_kernel(const TreeArgs a) {
    __shared__ int sums[kCombineThreads / 32];
    __shared__ int4 unit;                   // of the group at hand
    __shared__ int unit_w, unit_group;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int tid = threadIdx.x, c = tid >> 3;
    // thread i has worker i's task; what a task leads to lies in the workspace
    const int4 mine = tid < a.workers ? a.tasks[tid] : make_int4(-1, 0, 0, 0);
    const int parts_mine = mine.w & 0xff, lanes_mine = mine.w >> 8;
    const bool there = mine.x >= 0 && tid + (parts_mine - 1) * lanes_mine < a.workers;
    const int groups = there ? (mine.z * G + kCombineRows - 1) / kCombineRows : 0;
    int end = groups;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, end, off);
        if ((tid & 31) >= off) end += n;
    }
    if ((tid & 31) == 31) sums[tid >> 5] = end;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int k = 0; k < kCombineThreads / 32; ++k) {
        if (k < tid >> 5) end += sums[k];
        total += sums[k];
    }
#pragma unroll 1
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        if (item < end && item >= end - groups) {
            unit = mine;
            unit_w = tid;
            unit_group = item - (end - groups);
        }
        __syncthreads();
        const int4 task = unit;
        const int w = unit_w, r = unit_group * kCombineRows + (tid & 7);
        __syncthreads();
        const int parts = task.w & 0xff, lanes = task.w >> 8;
        const int tok = r / G, head = r % G;
        if (tok >= task.z || head >= a.group) continue;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < parts; i0 += kCombineBatch) {
            float2 e[kCombineBatch];
            float4 x[kCombineBatch];
#pragma unroll
            for (int k = 0; k < kCombineBatch; ++k) {
                const int i = i0 + k;
                if (i < parts) {
                    const int64_t slot = i == 0 ? 2 * w + 1 : 2 * (w + i * lanes);
                    e[k] = a.part_ml[slot * kPair + r];
                    x[k] = a.part_o[(slot * 32 + c) * kPair + r];
                }
            }
#pragma unroll
            for (int k = 0; k < kCombineBatch; ++k) {
                if (i0 + k >= parts || e[k].y == 0.f) continue;         // no token seen in the part
                const float mn = fmaxf(m, e[k].x);
                const float al = ex2(m - mn), be = ex2(e[k].x - mn);
                l = l * al + e[k].y * be;
                o.x = o.x * al + x[k].x * be;
                o.y = o.y * al + x[k].y * be;
                o.z = o.z * al + x[k].z * be;
                o.w = o.w * al + x[k].w * be;
                m = mn;
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t row = ((int64_t)task.x + tok) * a.num_q_heads + (int64_t)task.y * a.group + head;
        reinterpret_cast<uint2 *>(a.out)[row * 32 + c] =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    }
}

// q [total_q, Hq, 128] as (128, Hq, total_q) with boxes of 64 dims x G heads x
// box_rows(G) / G tokens.
bool make_q_map(CUtensorMap *m, const void *q, int total_q, int num_q_heads, int G) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)num_q_heads, (cuuint64_t)total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)kRowBytes, (cuuint64_t)num_q_heads * kRowBytes};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(box_rows(G) / G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_dependent(const void *fn, dim3 grid, unsigned block, size_t smem, void **args,
                             cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
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
cudaError_t launch_g(const TreeArgs &a, cudaStream_t st) {
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void *>(&tree_kernel<G>), kSmemBytes);
    if (e != cudaSuccess) return e;
    const int bs = 1 << a.block_size_log2;
    CUtensorMap mk, mv, mq;
    if (!make_box_map(&mk, a.k_cache, a.num_blocks, bs, a.num_kv_heads, a.head_major != 0, a.box_tokens) ||
        !make_box_map(&mv, a.v_cache, a.num_blocks, bs, a.num_kv_heads, a.head_major != 0, a.box_tokens) ||
        !make_q_map(&mq, a.q, a.total_q, a.num_q_heads, G))
        return cudaErrorInvalidValue;
    TreeArgs ac = a;
    void *args[] = {&ac, &mk, &mv, &mq};
    e = launch_dependent(reinterpret_cast<const void *>(&tree_kernel<G>), dim3((unsigned)a.workers), kThreads,
                         kSmemBytes, args, st);
    if (e != cudaSuccess) return e;
    return launch_dependent(reinterpret_cast<const void *>(&tree_combine_kernel<G>),
                            dim3((unsigned)(a.workers * kCombineCtas)), kCombineThreads, 0, args, st);
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

cudaError_t take_tree_error(cudaStream_t stream, int *code) {
    return take_device_word(g_tree_error, stream, code);
}

size_t tree_workspace_bytes(int workers) {
    const size_t slots = 2 * (size_t)workers * kPair;
    return round256((size_t)workers * sizeof(int4)) + slots * sizeof(float2) + slots * 32 * sizeof(float4);
}

void tree_carve_workspace(TreeArgs &a, void *workspace) {
    char *p = static_cast<char *>(workspace);
    const size_t slots = 2 * (size_t)a.workers * kPair;
    a.tasks = reinterpret_cast<int4 *>(p);
    p += round256((size_t)a.workers * sizeof(int4));
    a.part_ml = reinterpret_cast<float2 *>(p);
    a.part_o = reinterpret_cast<float4 *>(p + slots * sizeof(float2));
}

cudaError_t launch_decode_tree(const TreeArgs &a, int group_pad, cudaStream_t stream) {
    switch (group_pad) {
        case 1: return launch_g<1>(a, stream);
        case 2: return launch_g<2>(a, stream);
        case 4: return launch_g<4>(a, stream);
        case 8: return launch_g<8>(a, stream);
        case 16: return launch_g<16>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pa
