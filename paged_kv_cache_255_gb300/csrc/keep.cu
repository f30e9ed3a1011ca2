// Keeping the accepted tokens of drafts: of the n nodes at the end of a sequence those of
// one path stay, their cache rows moved to consecutive places in every pool, and the
// sequence gets shorter ("Implementation Details", Speculative Decoding -- EAGLE
// Proposer: of the drafted tokens the target model keeps those it agrees with).
//
// Place i takes the row of node kept[i]. The entries ascend, so kept[i] >= i, and a
// thread that moves its 16 bytes of all rows in the order of i never writes what it
// reads later: no second buffer, and no two threads touch the same bytes. The rows of a
// batch are read before they are written.
//
//   keep_kernel    a CTA takes 16-byte columns of all rows of one sequence; its threads
//                  look the rows up once
//   finish_kernel  a warp per sequence: the new length, and the blocks given back; a
//                  programmatic dependent, as the moves read both
//
// Bound by latency: list, table entry and row are three loads that wait for one another,
// and then the second launch: one layer of 4 sequences 6 us, 16 layers of 64 sequences (32
// pools, 21 MB read and written, 6.2 us of bytes) 14, the copy of the tables that the
// measurement needs included.
#include "common.cuh"
#include "keep_path.h"
#include "tree.h"

#include "../../include/pagedattn/decode_tree.h"

namespace pa {

__device__ int g_keep_error;         // first device-side error of a launch

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;                    // rows a thread has in flight
constexpr int kMaxKept = PA_KEEP_MAX_TOKENS;
constexpr int kFinishWarps = 4;
constexpr int kRowChunks = kHeadDim / 8;

__device__ __forceinline__ void set_error(int code) { atomicCAS(&g_keep_error, 0, code); }

// First token and nodes of sequence s's draft (0 nodes: nothing to do), and its length.
struct Draft {
    int first, n, L;
};
__device__ __forceinline__ Draft load_draft(const KeepArgs &a, int s) {
    const int64_t max_len = (int64_t)a.max_blocks << a.block_size_log2;
    const int64_t l = a.context_lens[s], L = l < 0 ? 0 : (l > max_len ? max_len : l);
    const int64_t q0 = a.starts[s], n = (int64_t)a.starts[s + 1] - q0;
    Draft d{0, 0, (int)L};
    if (q0 >= 0 && n > 0 && n <= L) {
        d.first = (int)(L - n);
        d.n = (int)n;
    }
    return d;
}
// Whether entry i of a list continues it; `bad` when it is no -1 either.
__device__ __forceinline__ bool continues(const int32_t *list, int i, int n, bool &bad) {
    return path_continues(__ldg(list + i), i == 0 ? 0 : __ldg(list + i - 1), i, n, bad);
}

__global__ void __launch_bounds__(kThreads) keep_kernel(const KeepArgs a, const PoolSet pools) {
    __shared__ int s_count;
    __shared__ int64_t s_from[kMaxKept], s_to[kMaxKept];    // rows of the pool, -1: not moved
    const int s = blockIdx.y, tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const Draft d = load_draft(a, s);
    if (d.n == 0) return;
    if (tid == 0) s_count = a.max_kept;
    __syncthreads();
    const int32_t *list = a.kept + (int64_t)s * a.max_kept;
    const int lb = a.block_size_log2;
    for (int i = tid; i < a.max_kept; i += kThreads) {
        bool bad;
        if (!continues(list, i, d.n, bad)) {
            atomicMin(&s_count, i);
            continue;
        }
        // Rows by token, or (head-major) by block, head 0, token. (An entry behind the list's end
        // that looks like one of a path is looked up too: its places are the draft's.)
        const int32_t *table = a.block_tables + (int64_t)s * a.max_blocks;
        auto row = [&](int t) -> int64_t {
            const int b = __ldg(table + (t >> lb));
            if (b <= 0 || b >= a.num_blocks) return -1;
            const int64_t off = t & ((1 << lb) - 1);
            return a.head_major ? (((int64_t)b * a.num_kv_heads) << lb) + off : (((int64_t)b << lb) + off) * a.num_kv_heads;
        };
        const int k = __ldg(list + i);
        int64_t from = row(d.first + k), to = row(d.first + i);
        if (k == i || from < 0 || to < 0) to = -1;
        s_from[i] = from;
        s_to[i] = to;
    }
    __syncthreads();
    const int count = s_count;
    const int per_pool = a.num_kv_heads * kRowChunks;
    const int64_t step = a.head_major ? (int64_t)kRowChunks << lb : kRowChunks;     // from a head to the next
    for (int64_t c = (int64_t)blockIdx.x * kThreads + tid; c < (int64_t)per_pool * pools.n; c += (int64_t)gridDim.x * kThreads) {
        const int pool = (int)(c / per_pool), col = (int)(c - (int64_t)pool * per_pool);
        uint4 *p = pools.p[pool] + (col / kRowChunks) * step + col % kRowChunks;
        for (int i0 = 0; i0 < count; i0 += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i0 + k < count && s_to[i0 + k] >= 0) x[k] = p[s_from[i0 + k] * kRowChunks];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i0 + k < count && s_to[i0 + k] >= 0) p[s_to[i0 + k] * kRowChunks] = x[k];
        }
    }
}

__global__ void __launch_bounds__(kFinishWarps * 32) finish_kernel(const KeepArgs a) {
    const int s = blockIdx.x * kFinishWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (s >= a.num_seqs) return;
    const Draft d = load_draft(a, s);
    if (d.n == 0) return;
    const int32_t *list = a.kept + (int64_t)s * a.max_kept;
    const int32_t *table = a.block_tables + (int64_t)s * a.max_blocks;
    const int lb = a.block_size_log2;
    int count = a.max_kept;
    for (int i0 = 0; i0 < a.max_kept; i0 += 32) {
        const int i = i0 + lane;
        bool bad = false;
        const bool ok = i < a.max_kept && continues(list, i, d.n, bad);
        const unsigned ends = __ballot_sync(0xffffffffu, i < a.max_kept && !ok);
        const int last = ends ? i0 + __ffs(ends) - 1 : i0 + 32;
        if (bad && i == last) set_error(kErrBadEntry);
        if (ok && i < last) {
            // (the moves have skipped it)
            const int k = __ldg(list + i);
            for (int t : {d.first + k, d.first + i}) {
                const int b = table[t >> lb];
                if (k != i && (b <= 0 || b >= a.num_blocks)) set_error(kErrBadEntry);
            }
        }
        if (ends) {
            count = last;
            break;
        }
    }
    __syncwarp();
    const int L = d.first + count;
    if (a.ref_counts) {
        const int first = (int)(((int64_t)L + (1 << lb) - 1) >> lb), end = (int)(((int64_t)d.L + (1 << lb) - 1) >> lb);
        int32_t *mine = a.block_tables + (int64_t)s * a.max_blocks;
        for (int e = first + lane; e < end; e += 32) {
            const int b = mine[e];
            mine[e] = 0;
            if (b == 0) continue;
            if (b < 0 || b >= a.num_blocks) {
                set_error(kErrBadEntry);
            } else if (atomicSub(a.ref_counts + b, 1) <= 0) {
                atomicAdd(a.ref_counts + b, 1);
                set_error(kErrBadEntry);
            }
        }
    }
    if (lane == 0) a.context_lens[s] = L;
}

template <class... Args>
cudaError_t launch_dependent(void (*fn)(Args...), dim3 grid, unsigned block, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

}  // namespace

cudaError_t take_keep_error(cudaStream_t stream, int *code) {
    return take_device_word(g_keep_error, stream, code);
}

cudaError_t launch_keep_tokens(void *const *caches, int num_caches, const KeepArgs &a, int sm_count,
                               cudaStream_t stream) {
    for (int i0 = 0; i0 < num_caches; i0 += kPoolsPerLaunch) {
        PoolSet pools{};
        pools.n = num_caches - i0 < kPoolsPerLaunch ? num_caches - i0 : kPoolsPerLaunch;
        for (int i = 0; i < pools.n; ++i) pools.p[i] = static_cast<uint4 *>(caches[i0 + i]);
        // as many CTAs a sequence as its columns need, or as fill the GPU
        const int64_t need = ((int64_t)a.num_kv_heads * kRowChunks * pools.n + kThreads - 1) / kThreads;
        const int64_t fair = ((int64_t)sm_count * 8 + a.num_seqs - 1) / a.num_seqs;
        const cudaError_t e = launch_dependent(keep_kernel, dim3((unsigned)(need < fair ? need : fair), (unsigned)a.num_seqs),
                                               kThreads, stream, a, pools);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(finish_kernel, dim3((unsigned)((a.num_seqs + kFinishWarps - 1) / kFinishWarps)),
                            kFinishWarps * 32, stream, a);
}

}  // namespace pa
