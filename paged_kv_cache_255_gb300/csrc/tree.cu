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
// space of all units' key tiles, and kUnitTiles places more a unit for what it costs
// besides them, is cut into equal contiguous shares, one CTA per SM each, planned by
// every CTA from the lengths and starts. A unit that one share holds whole is written
// as it ends; one that several share leaves a part per share in fp32, and
// tree_combine_kernel merges them by their running maxima and sums.
//
// Inside a CTA (TMEM: S_A 0-127, O_A 128-255, S_B 256-383, O_B 384-511 columns;
// P_t in bf16 over the first 64 columns of S_t):
//   warps 0-3, 4-7   softmax of query tile A, B: thread t owns row t (TMEM lane t);
//                    the mask's bits are read only on tiles that reach the nodes
//   warps 8, 9       K and V producers: TMA boxes of a block's tokens (16 .. 128) x 64
//                    dims; the V warp also loads the queries
//   warp 10          issues S = Q K^T and O += P V as their inputs arrive
//   warp 11          cleans V tiles that reach the nodes between their landing and their
//                    product: rows past the last token become 0, and so do infinities and
//                    NaN in nodes' rows (a weight of 0 times them is not 0). The rows that do see
//                    such a node add what was taken out after their result is written.
// Hand-offs are mbarriers; every wait is bounded (about 2 s), and a wait that ran out
// makes every role skip to its end. A role ends when what it has in flight has landed
// (or 0.1 s later); then the CTA frees its TMEM.
#include <climits>
#include <cmath>

#include "common.cuh"
#include "shared.h"
#include "tcgen05.cuh"
#include "tree.h"

namespace pa {

__device__ int g_tree_error;         // first device-side error of a launch

namespace {

constexpr int kRows = 128;                              // rows per query tile
constexpr int kPair = 2 * kRows;
constexpr int kKeys = 128;                              // keys per K/V tile
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kSoftmaxThreads = 256;
constexpr int kKWarp = kSoftmaxThreads / 32;            // 8
constexpr int kVWarp = kKWarp + 1;                      // 9
constexpr int kMmaWarp = kKWarp + 2;                    // 10
constexpr int kCleanWarp = kKWarp + 3;                  // 11
constexpr int kThreads = kSoftmaxThreads + 4 * 32;
constexpr int kWarpsAll = kThreads / 32;
constexpr int kGroup = 16;                              // tokens per MMA of P V
constexpr int kGroups = kKeys / kGroup;                 // 8
constexpr int kUnitPlaces = 2;                          // places of a unit besides its tiles
constexpr int kMinPlaces = 3;                           // fewest places of a share
constexpr int kMaskWords = 2 * 16;                      // 32-bit words of a mask row, at most
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
constexpr uint32_t kBarVLanded = kBarDrain + 1;          // + stage: a V tile that is to be cleaned
constexpr uint32_t kNumBars = kBarVLanded + kVStages;
constexpr uint32_t kOffTmemSlot = kOffCtl + 8 * kNumBars;
constexpr uint32_t kOffAbort = kOffTmemSlot + 4;
constexpr uint32_t kWalkBytes = 64;
constexpr uint32_t kOffWalk = (kOffAbort + 4 + 15) & ~15u;        // one Walk per warp
constexpr uint32_t kOffSums = kOffWalk + kWalkBytes * kWarpsAll;  // plan: a sum per warp
constexpr uint32_t kOffOdd = kOffSums + 8 * kWarpsAll;            // by parity of the piece: nodes whose V
constexpr uint32_t kOddBytes = 4 * (kMaskWords + 1);              // is not all finite, and whether any is
constexpr uint32_t kSmemBytes = kOffOdd + 2 * kOddBytes;
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescS = tc::idesc_bf16(128, kKeys, false);
constexpr uint32_t kIdescPV = tc::idesc_bf16(128, 128, true);
constexpr float kRescaleSlack = 8.f;                    // log2 units

__device__ __forceinline__ void set_error(int code) { atomicCAS(&g_tree_error, 0, code); }

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

// -- plan ------------------------------------------------------------------------

// A sequence's part of the work.
struct Seq {
    int q0, n, L;       // first query row, query rows (nodes), tokens
    int nt, pairs;      // key tiles; units of 256 query rows
};

template <int G>
__device__ __forceinline__ Seq load_seq(const TreeArgs &a, int s) {
    const int64_t max_len = (int64_t)a.max_blocks_per_seq << a.block_size_log2;     // below 2^31
    const int64_t l = __ldg(a.context_lens + s);
    int q0 = __ldg(a.starts + s), q1 = __ldg(a.starts + s + 1);
    q0 = q0 < 0 ? 0 : (q0 > a.total_q ? a.total_q : q0);
    q1 = q1 < q0 ? q0 : (q1 > a.total_q ? a.total_q : q1);
    Seq r;
    r.q0 = q0;
    r.n = q1 - q0;
    r.L = (int)(l < 0 ? 0 : (l > max_len ? max_len : l));
    r.nt = r.L > 0 ? (r.L + kKeys - 1) / kKeys : 1;     // an empty sequence's zeros are written by one tile
    r.pairs = (int)(((int64_t)r.n * G + kPair - 1) / kPair);
    return r;
}

__device__ __forceinline__ int64_t seq_places(const Seq &q, int num_kv_heads) {
    return (int64_t)q.pairs * num_kv_heads * (q.nt + kUnitPlaces);
}

// A share's walk over the flat space, sequence by sequence, KV head, pair, key tile: its
// pieces are runs of key tiles [j0, j1) of one unit. Every warp walks by itself and keeps
// its place in shared memory, where the fields are read when they are needed: none
// stays live across the tile loop.
struct alignas(16) Walk {
    int64_t T, T1;      // place of tile j0, end of the share
    Seq q;
    int s, kvh, pair, j0, j1;
};
static_assert(sizeof(Walk) == kWalkBytes, "Walk");

__device__ __forceinline__ void piece_end(Walk &w) {
    const int64_t left = w.T1 - w.T;
    w.j1 = w.q.nt - w.j0 < left ? w.q.nt : w.j0 + (int)left;
}

// On to the next unit; false at the end of the share.
template <int G>
__device__ __forceinline__ bool next_unit(Walk &w, const TreeArgs &a) {
    w.T += w.q.nt - w.j0 + kUnitPlaces;
    if (w.T >= w.T1) return false;
    w.j0 = 0;
    if (++w.pair == w.q.pairs) {
        w.pair = 0;
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
__device__ __forceinline__ bool walk_next(volatile Walk &place, const TreeArgs &a) {
    bool more = false;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) more = next_unit<G>(const_cast<Walk &>(place), a);
    more = __shfl_sync(0xffffffffu, more ? 1 : 0, 0) != 0;
    __syncwarp();
    return more;
}

// The total number of places, the shares in use, and this CTA's first piece (in
// `first`, shared memory); false when it has none. All threads call it.
template <int G>
__device__ __forceinline__ bool plan_share(const TreeArgs &a, Walk *first, volatile long long *sums,
                                           int64_t &W, int &shares) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = a.num_seqs, Hkv = a.num_kv_heads;
    Seq mine{};
    if (tid < S) mine = load_seq<G>(a, tid);
    long long local = tid < S ? seq_places(mine, Hkv) : 0;
    for (int s = tid + kThreads; s < S; s += kThreads) local += seq_places(load_seq<G>(a, s), Hkv);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) local += __shfl_xor_sync(0xffffffffu, local, m);
    if (lane == 0) sums[warp] = local;
    __syncthreads();
    W = 0;
    for (int i = 0; i < kWarpsAll; ++i) W += sums[i];
    __syncthreads();
    int64_t p = W / kMinPlaces;
    shares = (int)(p < 1 ? 1 : (p > a.workers ? a.workers : p));
    const int w = blockIdx.x;
    if (w >= shares || W == 0) return false;
    const int64_t T0 = (int64_t)w * W / shares, T1 = (int64_t)(w + 1) * W / shares;
    if (tid == 0) first->T1 = -1;               // nothing found yet
    int64_t base = 0;
    for (int c0 = 0; c0 < S && base <= T0; c0 += kThreads) {
        const int s = c0 + tid;
        const Seq q = c0 == 0 ? mine : (s < S ? load_seq<G>(a, s) : Seq{});
        const long long own = s < S ? seq_places(q, Hkv) : 0;
        long long v = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long n = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += n;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        long long before = base, end = base;
        for (int i = 0; i < kWarpsAll; ++i) {
            if (i < warp) before += sums[i];
            end += sums[i];
        }
        const long long excl = before + v - own;
        if (own > 0 && T0 >= excl && T0 < excl + own) {
            Walk k;
            const int64_t rem = T0 - excl;
            const int places = q.nt + kUnitPlaces;
            const int64_t unit = rem / places;
            k.T = T0;
            k.T1 = T1;
            k.q = q;
            k.s = s;
            k.kvh = (int)(unit / q.pairs);
            k.pair = (int)(unit - (int64_t)k.kvh * q.pairs);
            k.j0 = (int)(rem - unit * places);
            bool works = true;
            if (k.j0 >= q.nt) works = next_unit<G>(k, a);     // past the unit's tiles
            else piece_end(k);
            if (!works) k.T1 = -1;
            *first = k;
        }
        base = end;
        __syncthreads();
    }
    return first->T1 >= 0;
}

// -- masks -----------------------------------------------------------------------

// Bits [32 i, 32 i + 32) of a row of `words` mask words: nodes before the first (the
// context) are seen, those past the last are not.
__device__ __forceinline__ uint32_t mask_word(const uint32_t *row, int words, int i) {
    return i < 0 ? ~0u : (i < words ? row[i] : 0u);
}
// Of 32 nodes from node b on, those that exist (below n).
__device__ __forceinline__ uint32_t below(int n, int b) {
    const int k = n - b;
    return k <= 0 ? 0u : (k >= 32 ? ~0u : (1u << k) - 1u);
}

// Key tiles of a piece that a query tile (0 A, 1 B) computes: all, or none when the
// rows end before it.
template <int G>
__device__ __forceinline__ int piece_tiles(const volatile Walk &w, int t) {
    return w.pair * (kPair / G) + t * (kRows / G) < w.q.n ? w.j1 - w.j0 : 0;
}

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
// zero, and so do the elements of nodes' rows that are not finite; the nodes that had some
// are marked in `odd`. The 16-byte chunks of a row are permuted within it (128-byte
// swizzle), which does not matter here.
__device__ __forceinline__ void clean_v(const volatile Walk &w, int j, uint32_t vtile, uint32_t *odd, int words,
                                        int lane) {
    const int node0 = j * kKeys - (w.q.L - w.q.n);              // node of the tile's first key
    const int first = node0 < 0 ? -node0 : 0, left = w.q.L - j * kKeys;
    const int rows = groups_used(w, j) * kGroup - first;
#pragma unroll 4
    for (int i = lane; i < rows * 16; i += 32) {
        const int r = first + (i >> 4);
        const uint32_t at = vtile + ((i >> 3) & 1) * kKVHalf + r * 128 + (i & 7) * 16;
        uint32_t x[4] = {0u, 0u, 0u, 0u};
        bool store = true;
        if (r < left) {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"(at)
                         : "memory");
            store = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // an exponent of all ones: infinity or NaN
                const bool lo = (x[k] & 0x7f80u) == 0x7f80u, hi = (x[k] & 0x7f800000u) == 0x7f800000u;
                if (lo) x[k] &= 0xffff0000u;
                if (hi) x[k] &= 0x0000ffffu;
                store |= lo | hi;
            }
            const int node = node0 + r;
            if (store && node < 32 * words) {                   // the others nobody sees
                atomicOr(odd + (node >> 5), 1u << (node & 31));
                odd[kMaskWords] = 1u;
            }
        }
        if (store)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                         "r"(x[3])
                         : "memory");
    }
}

// What clean_v took out of the nodes that a row sees, added to its written result: the
// dims of those nodes that are not finite. `out` is the row in bf16, or `part` its words of
// a part in fp32. Rare.
__device__ __noinline__ void add_odd(const TreeArgs &a, const uint32_t *odd, int s, int kvh, int first_node,
                                     const uint32_t *mask_row, uint16_t *out, float4 *part) {
    const int lb = a.block_size_log2;
    for (int i = 0; i < a.mask_words; ++i)
        for (uint32_t bits = odd[i] & mask_row[i]; bits; bits &= bits - 1) {
            const int t = first_node + 32 * i + __ffs(bits) - 1;
            const int64_t bid = __ldg(a.block_tables + (int64_t)s * a.max_blocks_per_seq + (t >> lb));
            const int off = t & ((1 << lb) - 1);
            if (bid < 0 || bid >= a.num_blocks) continue;       // read as zeros
            const int64_t row = a.head_major ? ((bid * a.num_kv_heads + kvh) << lb) + off
                                             : ((bid << lb) + off) * a.num_kv_heads + kvh;
            const uint16_t *v = static_cast<const uint16_t *>(a.v_cache) + row * kHeadDim;
            for (int d = 0; d < kHeadDim; ++d) {
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

// -- attention ---------------------------------------------------------------------

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
tree_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap tmap_k,
            const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_q) {
    constexpr int BT = kRows / G;               // tokens per query tile
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
        tc::mbar_init(bar(kBarQFull), 1);
        tc::mbar_init(bar(kBarQEmpty), 1);
        for (int i = 0; i < kKStages; ++i) {
            tc::mbar_init(bar(kBarKFull + i), 1);
            tc::mbar_init(bar(kBarKEmpty + i), 1);
        }
        for (int i = 0; i < kVStages; ++i) {
            tc::mbar_init(bar(kBarVFull + i), 1);
            tc::mbar_init(bar(kBarVEmpty + i), 1);
            tc::mbar_init(bar(kBarVLanded + i), 1);
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

    // programmatic dependent of whatever precedes the call
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    int64_t W;
    int shares;
    Walk *walks = reinterpret_cast<Walk *>(smem + kOffWalk);
    const bool works = plan_share<G>(a, walks, reinterpret_cast<volatile long long *>(smem + kOffSums), W, shares);
    // the place of the first piece, for each warp its own
    {
        const Walk first = walks[0];
        __syncthreads();
        if ((tid & 31) == 0) walks[warp] = first;
        __syncwarp();
    }
    volatile Walk &w = walks[warp];
    const int w_id = blockIdx.x;
    if (warp == kVWarp && (tid & 31) == 0) a.tasks[w_id] = make_int4(-1, 0, 0, 0);
    if (!works) {
        // more CTAs than shares, or a share of no tiles
    } else if (tid < kSoftmaxThreads) {
        // ---------------- softmax warpgroups ----------------
        const int wg = tid >> 7, r = tid & 127;
        const uint32_t lane = (uint32_t)(r & ~31) << 16;
        const uint32_t tS = tmem + lane + wg * 256, tO = tS + 128;
        const float sc = a.scale_log2;
        // a masked score for the max: the value that loses whatever the scale's sign (masked
        // keys then get p = 0 directly)
        const float masked = sc >= 0.f ? -INFINITY : INFINITY;
        uint32_t gt = 0;                        // this query tile's key tiles before this piece
        int piece = 0;
        bool ok = true;
#pragma unroll 1
        do {
            const int ntt = piece_tiles<G>(w, wg);
            const int tok = w.pair * 2 * BT + wg * BT + r / G;
            const bool rv = tok < w.q.n && r % G < a.group;
            // warps past the last row only take part in the hand-offs
            const bool any = __any_sync(0xffffffffu, rv);
            float m = -INFINITY, lsum = 0.f;
#pragma unroll 1
            for (int j = 0; j < ntt; ++j) {
                const uint32_t gj = gt + j;
                const int kb = (w.j0 + j) * kKeys;
                const int b0 = kb - (w.q.L - w.q.n);            // node of the tile's first key
                const bool need_mask = any && b0 + kKeys > 0;
                uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
                if (need_mask) {
                    uint32_t mw[5] = {};
                    if (rv) {
                        const uint32_t *row = a.mask + ((int64_t)w.q.q0 + tok) * a.mask_words;
#pragma unroll
                        for (int k = 0; k < 5; ++k) mw[k] = mask_word(row, a.mask_words, (b0 >> 5) + k);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        vis[k] = __funnelshift_r(mw[k], mw[k + 1], b0 & 31) & below(w.q.n, b0 + 32 * k);
                }
                // S_t(j) done: also PV_t(j - 1), issued before it, so O is stable
                if (!warp_wait(bar(kBarSFull + wg), gj & 1, abort, true)) { ok = false; break; }
                tc::fence_after_sync();
                if (any) {
                    uint32_t sr[4][32];
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) tc::tmem_ld32(tS + ch * 32, sr[ch]);
                    tc::tmem_ld_wait();
                    if (need_mask) {
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(vis[ch] >> c & 1)) sr[ch][c] = __float_as_uint(masked);
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
                    // every score of the row masked: no new max (also for scale 0)
                    const float mt = ext == masked ? -INFINITY : ext * sc;
                    // the max is raised only when a tile exceeds it by 2^8: weights stay below
                    // 2^8, far inside fp32 and bf16 range, and O is rescaled rarely
                    bool rescale = false;
                    float alpha = 1.f;
                    if (mt > m + kRescaleSlack) {
                        rescale = m != -INFINITY;
                        alpha = rescale ? ex2(m - mt) : 1.f;
                        lsum *= alpha;
                        m = mt;
                    }
                    const float mb = m == -INFINITY ? 0.f : m;
                    // P = 2^(S sc - m), rounded to bf16 for the second product: its error of
                    // 2^-9 per weight averages out over the keys, and the output is rounded
                    // to bf16 as well
                    float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t pw[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            float p0 = ex2(fmaf(__uint_as_float(sr[ch][2 * c]), sc, -mb));
                            float p1 = ex2(fmaf(__uint_as_float(sr[ch][2 * c + 1]), sc, -mb));
                            if (need_mask) {
                                p0 = vis[ch] >> (2 * c) & 1 ? p0 : 0.f;
                                p1 = vis[ch] >> (2 * c + 1) & 1 ? p1 : 0.f;
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
                }
                tc::fence_before_sync();
                warp_arrive(bar(kBarPReady + wg));
            }
            if (!ok) break;
            if (ntt > 0) {
                if (!warp_wait(bar(kBarPVDone + wg), (gt + ntt - 1) & 1, abort, true)) { ok = false; break; }
                tc::fence_after_sync();
                if (any) {
                    const bool whole = w.j0 == 0 && w.j1 == w.q.nt;
                    // a row that saw nothing outputs zero, whatever its O
                    const float inv = whole ? 1.f / lsum : 1.f;
                    const int slot = 2 * w_id + (w.j0 == 0 ? 1 : 0);
                    float4 *po = a.part_o + (int64_t)slot * 32 * kPair + wg * kRows + r;
                    uint4 *orow = reinterpret_cast<uint4 *>(a.out) +
                                  (((int64_t)w.q.q0 + tok) * a.num_q_heads + (int64_t)w.kvh * a.group + r % G) * (kHeadDim / 8);
                    if (!whole && rv) a.part_ml[(int64_t)slot * kPair + wg * kRows + r] = make_float2(m, lsum);
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t o[32];
                        tc::tmem_ld32(tO + ch * 32, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o[c] = lsum == 0.f ? 0u : __float_as_uint(__uint_as_float(o[c]) * inv);
                        if (rv && whole) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const uint32_t *x = o + 8 * c;
                                auto f = [&](int i) { return __uint_as_float(x[i]); };
                                orow[ch * 4 + c] = make_uint4(pack_bf16x2(f(0), f(1)), pack_bf16x2(f(2), f(3)),
                                                              pack_bf16x2(f(4), f(5)), pack_bf16x2(f(6), f(7)));
                            }
                        } else if (rv) {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                po[(ch * 8 + c) * kPair] =
                                    make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                                __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
                        }
                    }
                    const uint32_t *odd = reinterpret_cast<const uint32_t *>(smem + kOffOdd + (piece & 1) * kOddBytes);
                    if (rv && reaches_nodes(w, w.j1 - 1) && odd[kMaskWords])
                        add_odd(a, odd, w.s, w.kvh, w.q.L - w.q.n, a.mask + ((int64_t)w.q.q0 + tok) * a.mask_words,
                                whole ? reinterpret_cast<uint16_t *>(orow) : nullptr, po);
                }
            }
            // (only after a piece that the tile took part in: nobody waits for the others)
            if (ntt > 0) {
                tc::fence_before_sync();
                warp_arrive(bar(kBarOFree + wg));
            }
            gt += ntt;
            ++piece;
        } while (walk_next<G>(w, a));
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
                                            w.kvh * a.group, w.q.q0 + w.pair * 2 * BT + t * BT, bar(kBarQFull));
                }
                warp_arrive(bar(kBarQFull));
                ++queries;
                // a unit that begins here and ends in another share: the combine's task
                if (lane == 0 && w.j0 == 0 && w.j1 < w.q.nt) {
                    const int64_t end = w.T + w.q.nt;           // past the unit's last tile
                    a.tasks[w_id] = make_int4(w.s, w.kvh, w.pair, (int)((end * shares - 1) / W));
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
                if (!warp_wait(bar_empty + 8 * st, ((gt / nst) & 1) ^ 1, abort)) { ok = false; break; }
                // a V tile that reaches the nodes is cleaned before it counts as there
                const uint32_t full = is_v && reaches_nodes(w, j) ? bar(kBarVLanded + st) : bar_full + 8 * st;
                const int n = __popc(__ballot_sync(0xffffffffu, at.x != INT_MIN));
                if (lane == 0) tc::mbar_expect_tx(full, (uint32_t)(n * box * 128));
                __syncwarp();
                if (at.x != INT_MIN)
                    tc::tma_load_3d(base + st * kKVBytes + h * kKVHalf + q * box * 128, map, h * 64, at.x, at.y, full);
                // the test hook holds back one V arrival (set_prefill_fault)
                if (!(is_v && a.fault_hold_v && gt == 0)) warp_arrive(full);
                ++gt;
            }
            ++piece;
        } while (ok && walk_next<G>(w, a));
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
        // In turn: PV_A(j), S_A(j + 1), PV_B(j), S_B(j + 1). PV_t(j) once P_t(j) is in TMEM
        // (and, for the first of a piece, the previous piece's O has been read); the tiles it
        // and S need have been waited for before, off the chain from P to S. A stage is
        // released after its last reader.
        uint32_t gt = 0, gq0 = 0, gq1 = 0;
        int piece = 0, pieces_b = 0;            // pieces before this one; those that had a tile B
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
                    if (ok && j == 0 && t == 0) {
                        // the results of the last piece of either tile are read (of B's also where
                        // this piece has no B: the marks of clean_v are free with them)
                        if (piece > 0) ok = await(bar(kBarOFree), (piece - 1) & 1);
                        if (ok && pieces_b > 0) ok = await(bar(kBarOFree + 1), (pieces_b - 1) & 1);
                    }
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
            pieces_b += two ? 1 : 0;
            ++piece;
        } while (ok && walk_next<G>(w, a));
        if (tc::elect_one()) tc::commit(bar(kBarDrain));
        __syncwarp();
        drain(bar(kBarDrain), 0);
    }

    if (works && warp == kCleanWarp) {
        // ---------------- cleaning of V tiles ----------------
        uint32_t gt = 0, landed = 0;                // tiles before this piece; bit i: parity of stage i's next phase
        int piece = 0;
        bool ok = true;
#pragma unroll 1
        do {
            bool fresh = true;
            uint32_t *odd = reinterpret_cast<uint32_t *>(smem + kOffOdd + (piece & 1) * kOddBytes);
#pragma unroll 1
            for (int j = w.j0; j < w.j1; ++j) {
                if (!reaches_nodes(w, j)) continue;
                const int st = (gt + (j - w.j0)) % kVStages;
                if (!warp_wait(bar(kBarVLanded + st), landed >> st & 1, abort)) { ok = false; break; }
                landed ^= 1u << st;
                if (fresh) {
                    // the V warp begins a piece once the products of the one before are done,
                    // and those wait for the results of the one before that: its marks are read
                    fresh = false;
                    for (int i = tid & 31; i <= kMaskWords; i += 32) odd[i] = 0u;
                    __syncwarp();
                }
                clean_v(w, j, sbase + kOffV + st * kKVBytes, odd, a.mask_words, tid & 31);
                tc::fence_proxy_async();
                warp_arrive(bar(kBarVFull + st));
            }
            gt += w.j1 - w.j0;
            ++piece;
        } while (ok && walk_next<G>(w, a));
    }

    // teardown: every role is done (or has given up) and has nothing in flight; TMEM is freed
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// Merge of the parts of the unit that worker blockIdx.x began and others ended: 8 rows
// x 32 words of 4 dims a CTA. A part's words are [dim / 4][row].
constexpr int kCombineRows = 8;
constexpr int kCombineBatch = 4;             // parts whose loads are in flight together

template <int G>
__global__ void __launch_bounds__(kCombineRows * 32) tree_combine_kernel(const TreeArgs a) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int w = blockIdx.x, r = blockIdx.y * kCombineRows + (threadIdx.x & 7), c = threadIdx.x >> 3;
    const int4 task = a.tasks[w];
    // after a wait that ran out the task may be of shares that wrote nothing; what is read lies in the workspace
    if (task.x < 0 || task.w <= w || task.w >= a.workers) return;
    const Seq q = load_seq<G>(a, task.x);
    const int tok = task.z * (kPair / G) + r / G, head = r % G;
    if (tok >= q.n || head >= a.group) return;
    const int parts = task.w - w + 1;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += kCombineBatch) {
        float2 e[kCombineBatch];
        float4 x[kCombineBatch];
#pragma unroll
        for (int k = 0; k < kCombineBatch; ++k) {
            const int i = i0 + k;
            if (i < parts) {
                const int64_t slot = i == 0 ? 2 * w + 1 : 2 * (w + i);
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
    const int64_t row = ((int64_t)q.q0 + tok) * a.num_q_heads + (int64_t)task.y * a.group + head;
    reinterpret_cast<uint2 *>(a.out)[row * 32 + c] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// q [total_q, Hq, 128] as (128, Hq, total_q) with boxes of 64 dims x G heads x 128 / G
// tokens: one half of a 128-row query tile.
bool make_q_map(CUtensorMap *m, const void *q, int total_q, int num_q_heads, int G) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)num_q_heads, (cuuint64_t)total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)kRowBytes, (cuuint64_t)num_q_heads * kRowBytes};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kRows / G)};
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
    const int64_t rows = (int64_t)a.total_q * G < kPair ? (int64_t)a.total_q * G : kPair;   // of a unit, at most
    return launch_dependent(reinterpret_cast<const void *>(&tree_combine_kernel<G>),
                            dim3((unsigned)a.workers, (unsigned)((rows + kCombineRows - 1) / kCombineRows)),
                            kCombineRows * 32, 0, args, st);
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
