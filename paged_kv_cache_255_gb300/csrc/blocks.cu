// Operations on the blocks of the paged cache: copy, fork, free, compact.
//
// A table row owns its first ceil(len / bs) entries ("Building a minimal vLLM
// implementation", sequence.py block_table); ref_counts[b] is the number of
// owned entries naming block b, and the free blocks are those with count 0.
// Block 0 is the null block, which is never owned, handed out or moved
// ("Implementation Details", PagedAttention -- BlockPool). All state is the
// caller's device memory, so a step that forks or frees needs no host round
// trip and can be captured in a graph.
//
// fork and compact run as two kernels:
//   plan   one cluster of 8 CTAs. Each of its warps owns a contiguous run
//          of block ids (and of forks), counts what it looks for with ballots,
//          and after one scan of the counts over the cluster's shared
//          memory walks its run again with the rank of each hit. The lowest
//          free ids come out in order, whatever the timing, with two reads of
//          the counts and no atomics.
//   apply  the whole GPU: table entries by thread, block data by warp. It is a
//          programmatic dependent of the plan and waits for its results.
// Block data moves in units of 4 KB (16 rows of 256 bytes: every block is a
// multiple of that), one warp per unit with all eight 16-byte loads of a lane
// in flight before its stores. Large calls are bound by HBM: 1819 blocks of
// 32 KB copied in 8 pools (of 2047 pairs, the others unused) take 148 us (6.5 TB/s
// read and written), a pool of 4096 such blocks, half of them live, is compacted
// in 89 us (6.0 TB/s); small ones by their launches: two blocks copied in
// 2.1 us, a pool of 128 compacted in 7.4 us. These and the times below are of a
// call within a graph of 20: the device's, without the host's.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace pa {

__device__ int g_blocks_error;       // first device-side error of a block operation

namespace {

constexpr int kPlanCtas = 8;                         // one cluster
// Warps of a plan CTA: each issues the whole plan, so few for small pools
// (32 warps: 2.4 us more over 128 blocks), many where reading the counts is most.
constexpr int kPlanFewWarps = 8;
constexpr int kPlanManyWarps = 32;
constexpr int64_t kPlanFewBlocks = 16384;            // 256 counts per warp
constexpr int kApplyThreads = 256;
constexpr int kApplyCtasPerSm = 8;
constexpr int kUnitChunks = 256;                     // 16-byte chunks of a 4 KB unit
constexpr int kLaneChunks = kUnitChunks / 32;
constexpr int kRowChunks = kHeadDim / 8;             // of one row of one KV head
constexpr int kSliceParts = 32;                      // 4 KB parts of a fork's copy a CTA takes together

__device__ __forceinline__ void set_error(int code) { atomicCAS(&g_blocks_error, 0, code); }

__device__ __forceinline__ int row_len(const int32_t *context_lens, int row, int64_t max_len) {
    const int64_t L = context_lens[row];
    return (int)(L < 0 ? 0 : (L > max_len ? max_len : L));
}

// What a warp's counts add up to over the cluster.
struct Scan {
    int before;     // sum of the counts of the warps before this one
    int total;
};

// Exclusive scan of one count per warp over the cluster's warps, in CTA then
// warp order. `mine` holds the CTA's counts; every thread of the cluster must
// call it, and `mine` may be reused after the next cluster sync.
template <int WARPS>
__device__ __forceinline__ Scan cluster_scan(cg::cluster_group &cl, int *mine, int count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) mine[warp] = count;
    cl.sync();
    Scan r{0, 0};
    const int self = (int)cl.block_rank() * WARPS + warp;
#pragma unroll
    for (int i = lane; i < kPlanCtas * WARPS; i += 32) {
        const int v = cl.map_shared_rank(mine, i / WARPS)[i % WARPS];
        r.total += v;
        r.before += i < self ? v : 0;
    }
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) {
        r.total += __shfl_xor_sync(0xffffffffu, r.total, x);
        r.before += __shfl_xor_sync(0xffffffffu, r.before, x);
    }
    return r;
}

// This warp's run [lo, hi) of n items, a multiple of 32 long but for the last.
template <int WARPS>
__device__ __forceinline__ void warp_run(int64_t n, int self, int64_t &lo, int64_t &hi) {
    constexpr int kAll = kPlanCtas * WARPS;
    const int64_t per = ((n + kAll - 1) / kAll + 31) & ~(int64_t)31;
    lo = per * self;
    hi = lo + per < n ? lo + per : n;
    lo = lo < n ? lo : n;
}

__device__ __forceinline__ unsigned lanes_below(int lane) { return (1u << lane) - 1u; }

// -- copying ------------------------------------------------------------------

// Up to 4 KB of a run of `n` 16-byte chunks, from chunk `c0` on.
__device__ __forceinline__ void copy_part(const uint4 *s, uint4 *d, int c0, int n, int lane) {
    uint4 v[kLaneChunks];
#pragma unroll
    for (int k = 0; k < kLaneChunks; ++k) {
        const int c = c0 + k * 32 + lane;
        if (c < n) v[k] = __ldcg(s + c);     // forks of one parent read the same rows
    }
#pragma unroll
    for (int k = 0; k < kLaneChunks; ++k) {
        const int c = c0 + k * 32 + lane;
        if (c < n) __stcs(d + c, v[k]);
    }
}

// A whole block is one run of full units: no index is checked.
__device__ __forceinline__ void copy_full_unit(uint4 *pool, int64_t src, int64_t dst, int unit,
                                               int block_chunks, int lane) {
    const uint4 *s = pool + src * block_chunks + unit * kUnitChunks + lane;
    uint4 *d = pool + dst * block_chunks + unit * kUnitChunks + lane;
    uint4 v[kLaneChunks];
#pragma unroll
    for (int k = 0; k < kLaneChunks; ++k) v[k] = __ldcs(s + k * 32);
#pragma unroll
    for (int k = 0; k < kLaneChunks; ++k) __stcs(d + k * 32, v[k]);
}

// Every warp of the grid takes units of the moves' data in turn.
__device__ __forceinline__ void move_all(const PoolSet &pools, const int2 *moves, int64_t n,
                                         int64_t num_blocks, int block_chunks, bool check) {
    const int lane = threadIdx.x & 31;
    const int units = block_chunks / kUnitChunks;
    const int64_t per_move = (int64_t)units * pools.n;
    const int64_t stride = (int64_t)gridDim.x * (kApplyThreads / 32);
    for (int64_t t = (int64_t)blockIdx.x * (kApplyThreads / 32) + (threadIdx.x >> 5);
         t < n * per_move; t += stride) {
        const int64_t i = t / per_move;
        const int r = (int)(t - i * per_move);
        const int pool = r / units;
        const int2 mv = moves[i];
        if (check) {
            if (mv.x == -1 || mv.y == -1) continue;
            if (mv.x < 0 || mv.y < 0 || mv.x >= num_blocks || mv.y >= num_blocks) {
                if (lane == 0) set_error(kErrBadEntry);
                continue;
            }
            if (mv.x == mv.y) continue;
        }
        copy_full_unit(pools.p[pool], mv.x, mv.y, r - pool * units, block_chunks, lane);
    }
}

__global__ void __launch_bounds__(kApplyThreads)
copy_blocks_kernel(const __grid_constant__ PoolSet pools, const int2 *pairs, int64_t num_pairs,
                   int64_t num_blocks, int block_chunks) {
    move_all(pools, pairs, num_pairs, num_blocks, block_chunks, true);
}

// -- free -----------------------------------------------------------------------
//
// Bound by its chain of dependent reads (row, length, entries, counts), and
// with many rows by the atomics on counts of far-apart blocks, one entry a thread
// in flight: 4 rows of 64 .. 1024 tokens take 3.5 us, 255 rows of 512 .. 16384 tokens
// (134800 blocks of 16) 12.0 us, both with the copy that restores the tables
// between passes.

// One reference to block b less. False when there was none to give up: the
// count is put back, so it ends at 0 however many such calls there were.
__device__ __forceinline__ bool drop_ref(int32_t *ref_counts, int b) {
    if (atomicSub(ref_counts + b, 1) > 0) return true;
    atomicAdd(ref_counts + b, 1);
    return false;
}

// One CTA per listed row. The row's length is taken and zeroed in one atomic
// exchange, so a row listed twice is freed once; counts are whole numbers, so
// the order of the atomics does not show.
__global__ void __launch_bounds__(kApplyThreads)
free_blocks_kernel(int32_t *block_tables, int max_blocks, int32_t *context_lens, int num_rows,
                   int32_t *ref_counts, const int32_t *rows, int block_size_log2,
                   int64_t num_blocks) {
    __shared__ int s_len;
    const int row = rows[blockIdx.x];
    if (row < 0 || row >= num_rows) {
        if (row != -1 && threadIdx.x == 0) set_error(kErrBadEntry);
        return;
    }
    if (threadIdx.x == 0) s_len = atomicExch(context_lens + row, 0);
    __syncthreads();
    const int64_t bs = (int64_t)1 << block_size_log2;
    const int64_t len = s_len < 0 ? 0 : s_len;
    const int64_t own = (len + bs - 1) >> block_size_log2;
    const int n = (int)(own < max_blocks ? own : max_blocks);
    int32_t *table = block_tables + (int64_t)row * max_blocks;
    for (int j = threadIdx.x; j < n; j += kApplyThreads) {
        const int b = table[j];
        table[j] = 0;
        if (b == 0) continue;
        if (b < 0 || b >= num_blocks || !drop_ref(ref_counts, b)) set_error(kErrBadEntry);
    }
}

// -- fork -------------------------------------------------------------------------

// What the plan decides for a fork: {parent row, tokens, rank of its new block
// among the free ones or -1, 0}; parent row -1 when the fork is skipped.
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) __cluster_dims__(kPlanCtas, 1, 1)
fork_plan_kernel(const ForkArgs a) {
    __shared__ int s_need[WARPS], s_free[WARPS];
    cg::cluster_group cl = cg::this_cluster();
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int self = (int)cl.block_rank() * WARPS + warp;
    const int64_t max_len = (int64_t)a.max_blocks << a.block_size_log2;

    int64_t f0, f1, b0, b1;
    warp_run<WARPS>(a.num_forks, self, f0, f1);
    warp_run<WARPS>(a.num_blocks, self, b0, b1);

    // a child may be forked once: the first fork that lists it gets it
    auto listed = [&a](int64_t i) {
        return a.parents[i] >= 0 && a.parents[i] < a.num_rows && a.children[i] >= 0 &&
               a.children[i] < a.num_rows;
    };
    for (int64_t i = f0 + lane; i < f1; i += 32)
        if (listed(i)) a.claim[a.children[i]] = 0x7fffffff;
    int nfree = 0;
#pragma unroll 4
    for (int64_t i = b0; i < b1; i += 32) {
        const int64_t b = i + lane;
        nfree += __popc(__ballot_sync(0xffffffffu, b > 0 && b < b1 && a.ref_counts[b] <= 0));
    }
    cl.sync();
    for (int64_t i = f0 + lane; i < f1; i += 32)
        if (listed(i)) atomicMin(a.claim + a.children[i], (int)i);
    cl.sync();

    int need = 0;
    for (int64_t i = f0; i < f1; i += 32) {
        bool tail = false;
        if (i + lane < f1) {
            const int p = a.parents[i + lane], c = a.children[i + lane];
            int4 r = make_int4(-1, 0, -1, 0);
            if (p == -1 || c == -1) {
                // an unused place in the list
            } else if (!listed(i + lane)) {
                set_error(kErrBadEntry);
            } else if (a.context_lens[c] > 0 || a.claim[c] != (int)(i + lane)) {
                set_error(kErrForkRefused);
            } else {
                r.x = p;
                r.y = row_len(a.context_lens, p, max_len);
                const int rows = r.y & ((1 << a.block_size_log2) - 1);
                if (rows > 0) {
                    // any other entry is passed on as it is: a block with count 0 is free, and
                    // may be another fork's new block while its rows would be read
                    const int b = a.block_tables[(int64_t)p * a.max_blocks + (r.y >> a.block_size_log2)];
                    tail = b > 0 && b < a.num_blocks && a.ref_counts[b] > 0;
                    if (b > 0 && b < a.num_blocks && !tail) set_error(kErrBadEntry);
                }
            }
            a.forks[i + lane] = r;
        }
        need += __popc(__ballot_sync(0xffffffffu, tail));
        if (tail) a.forks[i + lane].z = 0;      // marks the fork until its rank is known
    }
    const Scan sn = cluster_scan<WARPS>(cl, s_need, need);
    const Scan sf = cluster_scan<WARPS>(cl, s_free, nfree);

    int rank = sn.before;
    for (int64_t i = f0; i < f1; i += 32) {
        const bool tail = i + lane < f1 && a.forks[i + lane].z == 0;
        const unsigned m = __ballot_sync(0xffffffffu, tail);
        if (tail) {
            const int r = rank + __popc(m & lanes_below(lane));
            a.forks[i + lane].z = r;
            if (r >= sf.total) {                // no block left for it
                a.forks[i + lane].x = -1;
                set_error(kErrForkRefused);
            }
        }
        rank += __popc(m);
    }
    rank = sf.before;
    for (int64_t i = b0; i < b1 && rank < sn.total; i += 32) {
        const int64_t b = i + lane;
        const bool hit = b > 0 && b < b1 && a.ref_counts[b] <= 0;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        const int r = rank + __popc(m & lanes_below(lane));
        if (hit && r < sn.total) {
            // counted here, before any entry that names it adds to its count
            a.free_ids[r] = (int)b;
            a.ref_counts[b] = 1;
        }
        rank += __popc(m);
    }
    cl.sync();      // no CTA leaves while another may still read its counts
}

__global__ void __launch_bounds__(kApplyThreads)
fork_apply_kernel(const __grid_constant__ PoolSet pools, const ForkArgs a, int with_tables) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int bs_mask = (1 << a.block_size_log2) - 1;
    if (with_tables) {
        const int64_t stride = (int64_t)gridDim.x * kApplyThreads;
        for (int64_t t = (int64_t)blockIdx.x * kApplyThreads + threadIdx.x;
             t < (int64_t)a.num_forks * a.max_blocks; t += stride) {
            const int i = (int)(t / a.max_blocks), j = (int)(t - (int64_t)i * a.max_blocks);
            const int4 f = a.forks[i];
            if (f.x < 0) continue;
            const int c = a.children[i];
            if (j == 0) a.context_lens[c] = f.y;
            const int full = f.y >> a.block_size_log2;
            if (j >= full + ((f.y & bs_mask) != 0)) continue;
            int b = a.block_tables[(int64_t)f.x * a.max_blocks + j];
            if (j == full && f.z >= 0) b = a.free_ids[f.z];
            a.block_tables[(int64_t)c * a.max_blocks + j] = b;
            if (b != 0 && !(j == full && f.z >= 0)) {       // the plan has counted a new block
                if (b < 0 || b >= a.num_blocks || atomicAdd(a.ref_counts + b, 1) <= 0)
                    set_error(kErrBadEntry);    // passed on all the same
            }
        }
    }
    // The used rows of each parent's last block, into the child's new one: one
    // run in a token-major pool, one per KV head in a head-major one. A CTA
    // takes a slice of kSliceParts parts of up to 4 KB of one fork's block in
    // one pool. 256 forks of 16 parents, 8 pools, 512 KB blocks: 129 us, bound
    // by the writes of the new rows (569 MB at 4.4 TB/s; a parent's rows come from L2
    // after its first fork, 152 us when they were read past it). With a part per
    // warp and task, and a division for each of its chunks, it took 293 us.
    const int warp = threadIdx.x >> 5;
    const int slices = (a.block_chunks / kUnitChunks + kSliceParts - 1) / kSliceParts;
    const int64_t tasks = (int64_t)a.num_forks * pools.n * slices;
    for (int64_t t = blockIdx.x; t < tasks; t += gridDim.x) {
        const int64_t it = t / slices;
        const int slice = (int)(t - it * slices);
        const int i = (int)(it / pools.n), pool = (int)(it - (int64_t)i * pools.n);
        const int4 f = a.forks[i];
        if (f.x < 0 || f.z < 0) continue;
        const int used = f.y & bs_mask;
        const int run = a.head_major ? used * kRowChunks : used * a.num_kv_heads * kRowChunks;
        const int runs = a.head_major ? a.num_kv_heads : 1;
        const int per_run = (run + kUnitChunks - 1) / kUnitChunks;
        const int end = min((slice + 1) * kSliceParts, per_run * runs);
        if (slice * kSliceParts >= end) continue;
        const int64_t src = a.block_tables[(int64_t)f.x * a.max_blocks + (f.y >> a.block_size_log2)];
        const uint4 *s = pools.p[pool] + src * a.block_chunks;
        uint4 *d = pools.p[pool] + (int64_t)a.free_ids[f.z] * a.block_chunks;
        for (int part = slice * kSliceParts + warp; part < end; part += kApplyThreads / 32) {
            const int r = part / per_run, at = r * (bs_mask + 1) * kRowChunks;
            copy_part(s + at, d + at, (part - r * per_run) * kUnitChunks, run, lane);
        }
    }
}

// -- compact ------------------------------------------------------------------------

// With n live blocks, the k-th lowest live id above n moves to the k-th lowest
// free id up to n: the fewest moves that make the live ids 1 .. n, and no
// block is both read and written.
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) __cluster_dims__(kPlanCtas, 1, 1)
compact_plan_kernel(const CompactArgs a) {
    __shared__ int s_live[WARPS];
    __shared__ int s_low;               // live ids up to n, in the CTA that holds id n
    cg::cluster_group cl = cg::this_cluster();
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int self = (int)cl.block_rank() * WARPS + warp;
    int64_t b0, b1;
    warp_run<WARPS>(a.num_blocks, self, b0, b1);
    if (threadIdx.x == 0) s_low = 0;
    int live = 0;
#pragma unroll 4
    for (int64_t i = b0; i < b1; i += 32) {
        const int64_t b = i + lane;
        live += __popc(__ballot_sync(0xffffffffu, b > 0 && b < b1 && a.ref_counts[b] > 0));
    }
    const Scan s = cluster_scan<WARPS>(cl, s_live, live);
    const int n = s.total;
    if (n >= b0 && n < b1) {            // live ids up to n = live before this run, and in it up to n
        int low = s.before;
        for (int64_t i = b0; i <= n; i += 32) {
            const int64_t b = i + lane;
            low += __popc(__ballot_sync(0xffffffffu, b > 0 && b <= n && a.ref_counts[b] > 0));
        }
        if (lane == 0) s_low = low;
    }
    cl.sync();
    int low = 0;
    for (int c = 0; c < kPlanCtas; ++c) low += *cl.map_shared_rank(&s_low, c);
    if (self == 0 && lane == 0) {
        *a.num_moves = n - low;
        *a.num_live = n;
    }
    int rank = s.before;                // live ids before the 32 at hand
    for (int64_t i = b0; i < b1; i += 32) {
        const int64_t b = i + lane;
        const bool in = b > 0 && b < b1;
        const bool hit = in && a.ref_counts[b] > 0;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        const int before = rank + __popc(m & lanes_below(lane));
        if (hit && b > n) a.moves[before - low].x = (int)b;
        if (in && !hit && b <= n) a.moves[b - 1 - before].y = (int)b;
        if (b < b1 && (!hit || b <= n)) a.remap[b] = hit ? (int)b : 0;
        rank += __popc(m);
    }
    cl.sync();                          // the whole list is written; s_low has been read
    for (int k = self * 32 + lane; k < n - low; k += kPlanCtas * WARPS * 32) {
        const int2 mv = a.moves[k];
        a.remap[mv.x] = mv.y;
        a.ref_counts[mv.y] = a.ref_counts[mv.x];
        a.ref_counts[mv.x] = 0;
    }
}

__global__ void __launch_bounds__(kApplyThreads)
compact_apply_kernel(const __grid_constant__ PoolSet pools, const CompactArgs a, int with_tables) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (with_tables) {
        const int64_t max_len = (int64_t)a.max_blocks << a.block_size_log2;
        const int64_t stride = (int64_t)gridDim.x * kApplyThreads;
        for (int64_t t = (int64_t)blockIdx.x * kApplyThreads + threadIdx.x;
             t < (int64_t)a.num_rows * a.max_blocks; t += stride) {
            const int row = (int)(t / a.max_blocks), j = (int)(t - (int64_t)row * a.max_blocks);
            const int L = row_len(a.context_lens, row, max_len);
            if (((int64_t)j << a.block_size_log2) >= L) continue;
            const int b = a.block_tables[t];
            if (b == 0) continue;
            const int to = b > 0 && b < a.num_blocks ? a.remap[b] : 0;
            if (to == 0) {              // outside the pool, or a block nobody counts: left as it is
                set_error(kErrBadEntry);
            } else if (to != b) {
                a.block_tables[t] = to;
            }
        }
    }
    move_all(pools, a.moves, *a.num_moves, a.num_blocks, a.block_chunks, false);
}

// -- launches -------------------------------------------------------------------------

cudaError_t launch_dependent(const void *fn, unsigned grid, void **args, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kApplyThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// CTAs for `warps` warp-sized and `threads` thread-sized tasks, at most.
unsigned apply_grid(int64_t warps, int64_t threads, int sm_count) {
    const int64_t a = (warps + kApplyThreads / 32 - 1) / (kApplyThreads / 32);
    const int64_t b = (threads + kApplyThreads - 1) / kApplyThreads;
    int64_t n = a > b ? a : b;
    const int64_t most = (int64_t)sm_count * kApplyCtasPerSm;
    n = n < 1 ? 1 : n;
    return (unsigned)(n < most ? n : most);
}

// The pools, kPoolsPerLaunch at a time; once with none when there are none.
template <class F>
cudaError_t for_pools(void *const *caches, int num_caches, F &&launch) {
    for (int first = 0; first == 0 || first < num_caches; first += kPoolsPerLaunch) {
        PoolSet set{};
        set.n = num_caches - first < kPoolsPerLaunch ? num_caches - first : kPoolsPerLaunch;
        for (int i = 0; i < set.n; ++i) set.p[i] = static_cast<uint4 *>(caches[first + i]);
        const cudaError_t e = launch(set, first == 0);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace

cudaError_t take_blocks_error(cudaStream_t stream, int *code) {
    return take_device_word(g_blocks_error, stream, code);
}

// fork: a record per fork, a claim per row, at most num_rows new ids;
// compact: at most num_blocks / 2 moves and their count.
size_t blocks_workspace_bytes(int num_rows, int64_t num_blocks) {
    const size_t rows = (size_t)num_rows, moves = (size_t)(num_blocks / 2 + 1);
    const size_t fork = round16(rows * sizeof(int4)) + 2 * round16(rows * sizeof(int32_t));
    const size_t compact = 16 + round16(moves * sizeof(int2));
    return fork > compact ? fork : compact;
}

cudaError_t launch_copy_blocks(void *const *caches, int num_caches, const int32_t *pairs,
                               int64_t num_pairs, int64_t num_blocks, int block_chunks,
                               int sm_count, cudaStream_t stream) {
    return for_pools(caches, num_caches, [&](const PoolSet &set, bool) {
        const unsigned grid = apply_grid(num_pairs * set.n * (block_chunks / kUnitChunks), 0, sm_count);
        copy_blocks_kernel<<<grid, kApplyThreads, 0, stream>>>(
            set, reinterpret_cast<const int2 *>(pairs), num_pairs, num_blocks, block_chunks);
        return cudaGetLastError();
    });
}

cudaError_t launch_free_blocks(int32_t *block_tables, int max_blocks, int32_t *context_lens,
                               int num_rows, int32_t *ref_counts, const int32_t *rows, int num_freed,
                               int block_size_log2, int64_t num_blocks, cudaStream_t stream) {
    free_blocks_kernel<<<num_freed, kApplyThreads, 0, stream>>>(
        block_tables, max_blocks, context_lens, num_rows, ref_counts, rows, block_size_log2,
        num_blocks);
    return cudaGetLastError();
}

cudaError_t launch_fork_blocks(void *const *caches, int num_caches, ForkArgs a, void *workspace,
                               int sm_count, cudaStream_t stream) {
    char *w = static_cast<char *>(workspace);
    a.forks = reinterpret_cast<int4 *>(w);
    w += round16((size_t)a.num_rows * sizeof(int4));
    a.claim = reinterpret_cast<int32_t *>(w);
    w += round16((size_t)a.num_rows * sizeof(int32_t));
    a.free_ids = reinterpret_cast<int32_t *>(w);
    if (a.num_blocks <= kPlanFewBlocks)
        fork_plan_kernel<kPlanFewWarps><<<kPlanCtas, kPlanFewWarps * 32, 0, stream>>>(a);
    else
        fork_plan_kernel<kPlanManyWarps><<<kPlanCtas, kPlanManyWarps * 32, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return for_pools(caches, num_caches, [&](PoolSet set, bool first) {
        int with_tables = first ? 1 : 0;
        void *args[] = {&set, &a, &with_tables};
        const int64_t slices = (a.block_chunks / kUnitChunks + kSliceParts - 1) / kSliceParts;
        const unsigned grid = apply_grid((int64_t)a.num_forks * set.n * slices * (kApplyThreads / 32),
                                         first ? (int64_t)a.num_forks * a.max_blocks : 0, sm_count);
        return launch_dependent(reinterpret_cast<const void *>(&fork_apply_kernel), grid, args, stream);
    });
}

cudaError_t launch_compact_blocks(void *const *caches, int num_caches, CompactArgs a,
                                  void *workspace, int sm_count, cudaStream_t stream) {
    char *w = static_cast<char *>(workspace);
    a.num_moves = reinterpret_cast<int32_t *>(w);
    a.moves = reinterpret_cast<int2 *>(w + 16);
    if (a.num_blocks <= kPlanFewBlocks)
        compact_plan_kernel<kPlanFewWarps><<<kPlanCtas, kPlanFewWarps * 32, 0, stream>>>(a);
    else
        compact_plan_kernel<kPlanManyWarps><<<kPlanCtas, kPlanManyWarps * 32, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return for_pools(caches, num_caches, [&](PoolSet set, bool first) {
        int with_tables = first ? 1 : 0;
        void *args[] = {&set, &a, &with_tables};
        const unsigned grid = apply_grid(a.num_blocks / 2 * set.n * (a.block_chunks / kUnitChunks),
                                         first ? (int64_t)a.num_rows * a.max_blocks : 0, sm_count);
        return launch_dependent(reinterpret_cast<const void *>(&compact_apply_kernel), grid, args, stream);
    });
}

}  // namespace pa
