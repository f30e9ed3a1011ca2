// C ABI of libpagedattn: argument checks on the host, then kernel launches.
// The public contract is in include/pagedattn.h and include/pagedattn/.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "../../include/pagedattn.h"
#include "../../include/pagedattn/blocks.h"
#include "../../include/pagedattn/decode_shared.h"
#include "../../include/pagedattn/decode_tree.h"
#include "../../include/pagedattn/rotary.h"
#include "kernels.h"
#include "rotary.h"
#include "shared.h"
#include "tree.h"
#include "tree_plan.h"

namespace {

// One NVTX range per public call, named after the entry point, in the domain
// "libpagedattn": a timeline, or an Nsight Compute run filtered with --nvtx,
// shows which call launched each kernel. With no tool attached a push or a pop
// is a test of a function pointer.
nvtxDomainHandle_t trace_domain() {
    static const nvtxDomainHandle_t d = nvtxDomainCreateA("libpagedattn");
    return d;
}

class TraceRange {
  public:
    explicit TraceRange(const char *name) {
        nvtxEventAttributes_t a{};
        a.version = NVTX_VERSION;
        a.size = NVTX_EVENT_ATTRIB_STRUCT_SIZE;
        a.messageType = NVTX_MESSAGE_TYPE_ASCII;
        a.message.ascii = name;
        nvtxDomainRangePushEx(trace_domain(), &a);
    }
    ~TraceRange() { nvtxDomainRangePop(trace_domain()); }
    TraceRange(const TraceRange &) = delete;
    TraceRange &operator=(const TraceRange &) = delete;
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The TMA tile copies address the pool's rows with int32 coordinates: token
// rows (num_blocks * block_size) in the token-major map, (block, KV head)
// rows (num_blocks * num_kv_heads) in the head-major one.
bool pool_rows_fit(int64_t num_blocks, int block_size, int num_kv_heads) {
    return num_blocks * block_size < ((int64_t)1 << 31) &&
           num_blocks * num_kv_heads < ((int64_t)1 << 31);
}

int log2_exact(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return (1 << l) == x ? l : -1;
}

bool block_size_ok(int bs) { return bs >= 16 && bs <= 256 && log2_exact(bs) >= 0; }

// Per-device values the calls need on every launch, computed on a device's
// first call and kept: its SM count, and the decode's worker count for each
// padded group size (1, 2, 4, 8, 16) and tile kind (both depend only on the
// device and the kernels' resources). A racing first call computes the same
// value twice.
constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];
std::atomic<int> g_workers[kMaxDevices][5][2];

int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    return dev;
}

int current_sm_count() {
    const int dev = current_device();
    if (dev < 0) return 0;
    int n = g_sm_count[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    g_sm_count[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Comparison kernels kept for tests (pa_debug_kernel_variant); 0 = the
// product kernels. Read once per call, so a test that flips it between
// calls sees the change at the next call.
std::atomic<int> g_kernel_variant{0};

// Tile computation for decode: tensor cores, unless the test hook asks for
// the CUDA-core variant (single-token decode, group size <= 8).
pa::DecodeKernel decode_kernel_choice(int group_pad, int q_len) {
    if ((g_kernel_variant.load(std::memory_order_relaxed) & PA_VARIANT_DECODE_SIMT) &&
        group_pad <= 8 && q_len == 1)
        return pa::DecodeKernel::kSimt;
    return pa::DecodeKernel::kMma;
}

// Shares of the tile space for a call: forced, or from the device.
int plan_workers(int group_pad, pa::DecodeKernel k, int num_partitions) {
    if (num_partitions > 0) return num_partitions;
    const int dev = current_device();
    if (dev < 0) return 0;
    int gi = 0;
    while ((1 << gi) < group_pad && gi < 4) ++gi;
    std::atomic<int> &slot = g_workers[dev][gi][k == pa::DecodeKernel::kSimt ? 1 : 0];
    int P = slot.load(std::memory_order_relaxed);
    if (P > 0) return P;
    const int sms = current_sm_count();
    P = sms > 0 ? pa::decode_default_workers(group_pad, k, sms) : 0;
    if (P > 0) slot.store(P, std::memory_order_relaxed);
    return P;
}

// The arguments of a decode launch, but for the split and the workspace.
pa::DecodeArgs decode_args(const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, int q_len, float scale, void *out,
                           int num_seqs, int num_q_heads, int num_kv_heads, int block_size,
                           int64_t num_blocks, int layout) {
    pa::DecodeArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.out = out;
    a.num_seqs = num_seqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = num_q_heads / num_kv_heads;
    a.q_len = q_len;
    a.cols = a.group * q_len;
    a.block_size_log2 = log2_exact(block_size);
    a.head_major = layout == PA_LAYOUT_HEAD_MAJOR ? 1 : 0;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);   // scale * log2(e)
    return a;
}

pa_status_t decode_impl(const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *block_tables, int max_blocks_per_seq,
                        const int32_t *context_lens, int q_len, float scale, void *out,
                        int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                        int block_size, int64_t num_blocks, int layout, void *workspace,
                        size_t workspace_bytes, int num_partitions, void *stream,
                        bool plan_early = false) {
    bool nothing_to_do = false;
    const pa_status_t chk = pa::decode_check_args(
        q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, q_len, scale, out,
        num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, layout,
        num_partitions, &nothing_to_do);
    if (chk != PA_OK || nothing_to_do) return chk;
    const int gp = pa::decode_group_pad(num_q_heads / num_kv_heads * q_len);

    const pa::DecodeKernel kind = decode_kernel_choice(gp, q_len);
    const int P = plan_workers(gp, kind, num_partitions);
    if (P <= 0) return PA_ERR_CUDA;
    if (!workspace || !aligned16(workspace) || workspace_bytes < pa::decode_workspace_bytes(gp, P))
        return PA_ERR_WORKSPACE;

    pa::DecodeArgs a = decode_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                   context_lens, q_len, scale, out, num_seqs, num_q_heads,
                                   num_kv_heads, block_size, num_blocks, layout);
    a.num_workers = P;
    a.min_tiles = num_partitions > 0 ? 1 : pa::kDefaultMinTiles;
    a.plan_early = plan_early ? 1 : 0;
    pa::decode_carve_workspace(a, workspace, gp);
    const cudaError_t e = pa::launch_decode(a, gp, kind, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t store_impl(const void *k, const void *v, void *k_cache, void *v_cache,
                       const int64_t *slot_mapping, int64_t num_tokens, int num_kv_heads,
                       int head_dim, int block_size, int64_t num_blocks, int layout,
                       void *stream) {
    bool nothing_to_do = false;
    const pa_status_t chk = pa::store_check_args(k, v, k_cache, v_cache, slot_mapping, num_tokens,
                                                 num_kv_heads, head_dim, block_size, num_blocks,
                                                 layout, &nothing_to_do);
    if (chk != PA_OK || nothing_to_do) return chk;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const cudaError_t e = pa::launch_store_kvcache(
        k, v, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim,
        log2_exact(block_size), num_blocks * block_size, layout == PA_LAYOUT_HEAD_MAJOR ? 1 : 0,
        sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t prefill_impl(const void *q, const void *k_cache, const void *v_cache,
                         const int32_t *block_tables, int max_blocks_per_seq,
                         const int32_t *context_lens, const int32_t *query_start_loc,
                         int max_query_len, float scale, void *out, int num_seqs, int total_q,
                         int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                         int64_t num_blocks, int layout, void *stream) {
    if (layout != PA_LAYOUT_TOKEN_MAJOR && layout != PA_LAYOUT_HEAD_MAJOR) return PA_ERR_INVALID_ARG;
    if (num_seqs < 0 || total_q < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_blocks < 0 || max_blocks_per_seq < 0 || max_query_len < 0 || !std::isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    if (head_dim != pa::kHeadDimPublic || !block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
    const int group = num_q_heads / num_kv_heads;
    const int gp = pa::decode_group_pad(group);
    if (gp == 0) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start_loc || !out)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return PA_ERR_INVALID_ARG;
    if (max_blocks_per_seq == 0 || num_blocks == 0) return PA_ERR_INVALID_ARG;
    if (num_seqs > 65535 || num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (!pool_rows_fit(num_blocks, block_size, num_kv_heads)) return PA_ERR_UNSUPPORTED;
    pa::PrefillArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start_loc = query_start_loc;
    a.out = out;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = group;
    a.block_size_log2 = log2_exact(block_size);
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.head_major = layout == PA_LAYOUT_HEAD_MAJOR ? 1 : 0;
    a.fault_hold_v = pa::prefill_fault();
    a.num_blocks = num_blocks;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    const int mql = max_query_len > 0 ? max_query_len : 1;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool mma = g_kernel_variant.load(std::memory_order_relaxed) & PA_VARIANT_PREFILL_MMA;
    const cudaError_t e = mma ? pa::launch_prefill(a, gp, mql, st)
                              : pa::launch_prefill_tc(a, gp, mql, st);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Columns of the decode tiles of a call over shared prefixes.
int shared_cols(int group_pad) { return group_pad <= 8 ? 8 : 16; }

// The shape of the pools a block operation works on, and their addresses.
pa_status_t check_pools(void *const *caches, int num_caches, int num_kv_heads, int head_dim,
                        int block_size, int64_t num_blocks) {
    if (num_caches < 0 || num_kv_heads <= 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
    if (head_dim != pa::kHeadDimPublic || !block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
    if (num_kv_heads > 65535 || num_blocks > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (num_caches > 0 && !caches) return PA_ERR_INVALID_ARG;
    for (int i = 0; i < num_caches; ++i)
        if (!caches[i] || !aligned16(caches[i])) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

int block_chunks_of(int num_kv_heads, int head_dim, int block_size) {
    return block_size * num_kv_heads * (head_dim / 8);
}

pa_status_t check_workspace(const void *workspace, size_t workspace_bytes, int num_rows,
                            int64_t num_blocks) {
    const bool ok = workspace && aligned16(workspace) &&
                    workspace_bytes >= pa::blocks_workspace_bytes(num_rows, num_blocks);
    return ok ? PA_OK : PA_ERR_WORKSPACE;
}

// Rows of `heads` heads of `tokens` tokens: address, and the strides that are used.
bool rows_ok(const void *p, int64_t tokens, int64_t token, int heads, int64_t head) {
    auto ok = [](int64_t n, int64_t stride) { return n <= 1 || (stride >= 0 && stride % 8 == 0); };
    return p && aligned16(p) && ok(tokens, token) && ok(heads, head);
}

// Whether an output's rows lie apart: heads inside tokens, or tokens inside heads.
bool rows_apart(int64_t tokens, int64_t token, int heads, int64_t head) {
    const int64_t D = pa::kHeadDimPublic;
    if (tokens <= 1) return heads <= 1 || head >= D;
    if (heads <= 1) return token >= D;
    const bool heads_inside = head <= token;
    const int64_t in = heads_inside ? head : token, out = heads_inside ? token : head;
    const int64_t n = heads_inside ? heads : tokens;
    return in >= D && (out - D) / in >= n - 1;      // out >= (n - 1) in + D
}

// What pa_rotate and pa_append_kvcache check alike, and the arguments of a launch.
pa_status_t rotate_args(pa::RotateArgs &a, bool *interleaved, const void *q, int64_t q_token,
                        int64_t q_head, void *q_out, int64_t qo_token, int64_t qo_head,
                        int num_q_heads, const void *k, int64_t k_token, int64_t k_head,
                        int num_kv_heads, int head_dim, const int32_t *positions,
                        int64_t num_tokens, const pa_rotary_t *rotary, const void *q_weight,
                        const void *k_weight, float eps) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || !std::isfinite(eps) || eps < 0.f)
        return PA_ERR_INVALID_ARG;
    if (head_dim != pa::kHeadDimPublic) return PA_ERR_UNSUPPORTED;
    if ((int64_t)num_q_heads + num_kv_heads > (1 << 20) || num_tokens > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (rotary) {
        if (!std::isfinite(rotary->amplitude)) return PA_ERR_INVALID_ARG;
        if (rotary->rot_dim < 16 || rotary->rot_dim > head_dim || rotary->rot_dim % 16 != 0)
            return PA_ERR_UNSUPPORTED;
    }
    if (num_tokens == 0) return PA_OK;
    if (rotary && !positions) return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!rows_ok(q, num_tokens, q_token, num_q_heads, q_head) ||
                            !rows_ok(q_out, num_tokens, qo_token, num_q_heads, qo_head) ||
                            !rows_apart(num_tokens, qo_token, num_q_heads, qo_head)))
        return PA_ERR_INVALID_ARG;
    if (num_kv_heads > 0 && !rows_ok(k, num_tokens, k_token, num_kv_heads, k_head)) return PA_ERR_INVALID_ARG;
    if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)))
        return PA_ERR_INVALID_ARG;
    a.q = {static_cast<const uint4 *>(q), q_token / 8, q_head / 8};
    a.k = {static_cast<const uint4 *>(k), k_token / 8, k_head / 8};
    a.q_out = {static_cast<uint4 *>(q_out), qo_token / 8, qo_head / 8};
    a.positions = rotary ? positions : nullptr;
    a.q_weight = static_cast<const uint4 *>(q_weight);
    a.k_weight = static_cast<const uint4 *>(k_weight);
    a.num_tokens = num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.eps = eps;
    *interleaved = rotary && rotary->interleaved;
    if (rotary) {
        a.pairs = rotary->rot_dim / 2;
        a.amplitude = rotary->amplitude;
        for (int i = 0; i < a.pairs; ++i) a.turns[i] = rotary->turns[i];
    }
    return PA_OK;
}

}  // namespace

namespace pa {

pa_status_t store_check_args(const void *k, const void *v, const void *k_cache,
                             const void *v_cache, const int64_t *slot_mapping, int64_t num_tokens,
                             int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                             int layout, bool *nothing_to_do) {
    *nothing_to_do = false;
    if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks < 0) return PA_ERR_INVALID_ARG;
    if (layout != PA_LAYOUT_TOKEN_MAJOR && layout != PA_LAYOUT_HEAD_MAJOR) return PA_ERR_INVALID_ARG;
    if (head_dim != kHeadDimPublic || !block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) {
        *nothing_to_do = true;
        return PA_OK;
    }
    if (!k || !v || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

pa_status_t decode_check_args(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_tables, int max_blocks_per_seq,
                              const int32_t *context_lens, int q_len, float scale,
                              const void *out, int num_seqs, int num_q_heads, int num_kv_heads,
                              int head_dim, int block_size, int64_t num_blocks, int layout,
                              int num_partitions, bool *nothing_to_do) {
    *nothing_to_do = false;
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks < 0 ||
        max_blocks_per_seq < 0 || num_partitions < 0 || q_len < 1 || !std::isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    if (layout != PA_LAYOUT_TOKEN_MAJOR && layout != PA_LAYOUT_HEAD_MAJOR) return PA_ERR_INVALID_ARG;
    if (head_dim != kHeadDimPublic || !block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
    const int group = num_q_heads / num_kv_heads;
    if (q_len > 16) return PA_ERR_UNSUPPORTED;
    if (decode_group_pad(group * q_len) == 0) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) {
        *nothing_to_do = true;
        return PA_OK;
    }
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return PA_ERR_INVALID_ARG;
    if (max_blocks_per_seq == 0 || num_blocks == 0) return PA_ERR_INVALID_ARG;
    if (!pool_rows_fit(num_blocks, block_size, num_kv_heads)) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

}  // namespace pa

extern "C" {

const char *pa_status_string(pa_status_t status) {
    switch (status) {
        case PA_OK: return "PA_OK";
        case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
        case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
        case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE";
        case PA_ERR_CUDA: return "PA_ERR_CUDA";
    }
    return "PA_ERR_UNKNOWN";
}

pa_status_t pa_store_kvcache_layout(const void *k, const void *v, void *k_cache, void *v_cache,
                                    const int64_t *slot_mapping, int64_t num_tokens,
                                    int num_kv_heads, int head_dim, int block_size,
                                    int64_t num_blocks, pa_layout_t layout, void *stream) {
    TraceRange r("pa_store_kvcache_layout");
    return store_impl(k, v, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim,
                      block_size, num_blocks, layout, stream);
}

pa_status_t pa_store_kvcache(const void *k, const void *v, void *k_cache, void *v_cache,
                             const int64_t *slot_mapping, int64_t num_tokens, int num_kv_heads,
                             int head_dim, int block_size, int64_t num_blocks, void *stream) {
    TraceRange r("pa_store_kvcache");
    return store_impl(k, v, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim,
                      block_size, num_blocks, PA_LAYOUT_TOKEN_MAJOR, stream);
}

size_t pa_decode_workspace_size(int num_q_heads, int num_kv_heads, int head_dim,
                                int num_partitions) {
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        head_dim != pa::kHeadDimPublic || num_partitions < 0)
        return 0;
    const int gp = pa::decode_group_pad(num_q_heads / num_kv_heads);
    if (gp == 0) return 0;
    // sized for the larger of the two variants' default share counts
    int P = plan_workers(gp, pa::DecodeKernel::kMma, num_partitions);
    if (num_partitions == 0 && gp <= 8) {
        const int Ps = plan_workers(gp, pa::DecodeKernel::kSimt, 0);
        P = Ps > P ? Ps : P;
    }
    if (P <= 0) return 0;
    return pa::decode_workspace_bytes(gp, P);
}

pa_status_t pa_decode(const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_tables, int max_blocks_per_seq,
                      const int32_t *context_lens, float scale, void *out, int num_seqs,
                      int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                      int64_t num_blocks, void *workspace, size_t workspace_bytes,
                      void *stream) {
    TraceRange r("pa_decode");
    return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, 1,
                       scale, out, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, PA_LAYOUT_TOKEN_MAJOR, workspace, workspace_bytes, 0, stream);
}

pa_status_t pa_decode_splitk(const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, int max_blocks_per_seq,
                             const int32_t *context_lens, float scale, void *out, int num_seqs,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             int64_t num_blocks, void *workspace, size_t workspace_bytes,
                             int num_partitions, void *stream) {
    TraceRange r("pa_decode_splitk");
    if (num_partitions < 0) return PA_ERR_INVALID_ARG;
    return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, 1,
                       scale, out, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, PA_LAYOUT_TOKEN_MAJOR, workspace, workspace_bytes,
                       num_partitions, stream);
}

size_t pa_decode_multi_workspace_size(int q_len, int num_q_heads, int num_kv_heads,
                                      int head_dim) {
    if (q_len < 1 || q_len > 16 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_q_heads % num_kv_heads != 0 || head_dim != pa::kHeadDimPublic)
        return 0;
    const int gp = pa::decode_group_pad(num_q_heads / num_kv_heads * q_len);
    if (gp == 0) return 0;
    const int P = plan_workers(gp, pa::DecodeKernel::kMma, 0);
    return P > 0 ? pa::decode_workspace_bytes(gp, P) : 0;
}

pa_status_t pa_decode_layout(const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, int max_blocks_per_seq,
                             const int32_t *context_lens, float scale, void *out, int num_seqs,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             int64_t num_blocks, pa_layout_t layout, void *workspace,
                             size_t workspace_bytes, int num_partitions, void *stream) {
    TraceRange r("pa_decode_layout");
    if (num_partitions < 0) return PA_ERR_INVALID_ARG;
    return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, 1,
                       scale, out, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, layout, workspace, workspace_bytes, num_partitions, stream);
}

pa_status_t pa_decode_multi(const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *block_tables, int max_blocks_per_seq,
                            const int32_t *context_lens, int q_len, float scale, void *out,
                            int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                            int block_size, int64_t num_blocks, void *workspace,
                            size_t workspace_bytes, void *stream) {
    TraceRange r("pa_decode_multi");
    return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                       q_len, scale, out, num_seqs, num_q_heads, num_kv_heads, head_dim,
                       block_size, num_blocks, PA_LAYOUT_TOKEN_MAJOR, workspace,
                       workspace_bytes, 0, stream);
}

pa_status_t pa_decode_multi_layout(const void *q, const void *k_cache, const void *v_cache,
                                   const int32_t *block_tables, int max_blocks_per_seq,
                                   const int32_t *context_lens, int q_len, float scale, void *out,
                                   int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                   int block_size, int64_t num_blocks, pa_layout_t layout,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    TraceRange r("pa_decode_multi_layout");
    return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                       q_len, scale, out, num_seqs, num_q_heads, num_kv_heads, head_dim,
                       block_size, num_blocks, layout, workspace, workspace_bytes, 0, stream);
}

pa_status_t pa_decode_step(const void *k, const void *v, const int64_t *slot_mapping,
                           int64_t num_tokens, const void *q, void *k_cache, void *v_cache,
                           const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, float scale, void *out, int num_seqs,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int64_t num_blocks, pa_layout_t layout, void *workspace,
                           size_t workspace_bytes, void *stream) {
    TraceRange r("pa_decode_step");
    // every argument of both calls is checked before anything is launched
    bool no_store = false, no_decode = false;
    pa_status_t chk = pa::store_check_args(k, v, k_cache, v_cache, slot_mapping, num_tokens,
                                           num_kv_heads, head_dim, block_size, num_blocks, layout,
                                           &no_store);
    if (chk != PA_OK) return chk;
    chk = pa::decode_check_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                context_lens, 1, scale, out, num_seqs, num_q_heads, num_kv_heads,
                                head_dim, block_size, num_blocks, layout, 0, &no_decode);
    if (chk != PA_OK) return chk;
    if (!no_decode) {
        const int gp = pa::decode_group_pad(num_q_heads / num_kv_heads);
        const int P = plan_workers(gp, decode_kernel_choice(gp, 1), 0);
        if (P <= 0) return PA_ERR_CUDA;
        if (!workspace || !aligned16(workspace) ||
            workspace_bytes < pa::decode_workspace_bytes(gp, P))
            return PA_ERR_WORKSPACE;
    }
    chk = store_impl(k, v, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim,
                     block_size, num_blocks, layout, stream);
    if (chk != PA_OK) return chk;
    // with the store just queued, the decode plans its split while the store runs
    return decode_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, 1,
                       scale, out, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, layout, workspace, workspace_bytes, 0, stream, !no_store);
}

size_t pa_decode_shared_workspace_size(int num_seqs, int num_groups, int num_q_heads,
                                       int num_kv_heads, int head_dim) {
    if (num_seqs < 0 || num_groups < 0 || num_groups > pa::kSharedMaxGroups || num_seqs > 65535 ||
        num_kv_heads > 65535)
        return 0;
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        head_dim != pa::kHeadDimPublic)
        return 0;
    const int gp = pa::decode_group_pad(num_q_heads / num_kv_heads);
    if (gp == 0) return 0;
    const int P = plan_workers(shared_cols(gp), pa::DecodeKernel::kMma, 0), sms = current_sm_count();
    if (P <= 0 || sms <= 0) return 0;
    return round256(pa::decode_workspace_bytes(shared_cols(gp), P)) +
           pa::shared_workspace_bytes(num_seqs, num_groups, num_q_heads, num_kv_heads, gp, sms);
}

pa_status_t pa_decode_shared(const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, int max_blocks_per_seq,
                             const int32_t *context_lens, const int32_t *group_starts,
                             const int32_t *prefix_blocks, int num_groups, float scale, void *out,
                             int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                             int block_size, int64_t num_blocks, pa_layout_t layout,
                             void *workspace, size_t workspace_bytes, void *stream) {
    TraceRange r("pa_decode_shared");
    if (num_groups < 0) return PA_ERR_INVALID_ARG;
    bool nothing_to_do = false;
    const pa_status_t chk = pa::decode_check_args(
        q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, 1, scale, out, num_seqs,
        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, layout, 0, &nothing_to_do);
    if (chk != PA_OK) return chk;
    if (num_groups > pa::kSharedMaxGroups || num_seqs > 65535 || num_kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    // tokens are counted in 32 bits, rounded up to tiles of 128
    if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX - 127) return PA_ERR_UNSUPPORTED;
    if (nothing_to_do || num_groups == 0) return PA_OK;
    if (!group_starts || !prefix_blocks) return PA_ERR_INVALID_ARG;
    const int gp = pa::decode_group_pad(num_q_heads / num_kv_heads);
    const int P = plan_workers(shared_cols(gp), pa::DecodeKernel::kMma, 0);
    const int sms = current_sm_count();
    if (P <= 0 || sms <= 0) return PA_ERR_CUDA;
    const size_t dec = round256(pa::decode_workspace_bytes(shared_cols(gp), P));
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < dec + pa::shared_workspace_bytes(num_seqs, num_groups, num_q_heads,
                                                           num_kv_heads, gp, sms))
        return PA_ERR_WORKSPACE;
    pa::DecodeArgs a = decode_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                   context_lens, 1, scale, out, num_seqs, num_q_heads, num_kv_heads,
                                   block_size, num_blocks, layout);
    a.num_workers = P;
    a.min_tiles = pa::kDefaultMinTiles;
    pa::decode_carve_workspace(a, workspace, shared_cols(gp));
    pa::SharedArgs sh{};
    sh.group_starts = group_starts;
    sh.prefix_blocks = prefix_blocks;
    sh.num_groups = num_groups;
    sh.group_pad = gp;
    sh.max_workers = sms;
    sh.box_tokens = block_size < 128 ? block_size : 128;
    // Where one packed unit takes every sequence, it is never dearer than the
    // prefix kernel, which is then not launched. Nor is it where its tiles could not be
    // counted in 32 bits, or for a scale that is not positive, which it does not
    // take (every sequence then reads its prefix by itself, or packed).
    const int64_t key_tiles = (((int64_t)max_blocks_per_seq << a.block_size_log2) + 127) / 128;
    const int64_t pairs = (int64_t)num_seqs * gp / pa::kPairRows + num_groups;
    sh.tensor = (num_seqs + pa::shared_fit(a.group) - 1) / pa::shared_fit(a.group) > 1 &&
                key_tiles <= INT32_MAX / num_kv_heads / pairs && a.scale_log2 > 0.f && sms > 1 ? 1 : 0;
    sh.fault_hold_v = pa::prefill_fault();
    pa::shared_carve_workspace(sh, static_cast<char *>(workspace) + dec, a);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = pa::launch_shared_prefix(a, sh, st);
    if (e == cudaSuccess) e = pa::launch_decode_shared(a, sh, st);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t pa_prefill(const void *q, const void *k_cache, const void *v_cache,
                       const int32_t *block_tables, int max_blocks_per_seq,
                       const int32_t *context_lens, const int32_t *query_start_loc,
                       int max_query_len, float scale, void *out, int num_seqs, int total_q,
                       int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                       int64_t num_blocks, void *stream) {
    TraceRange r("pa_prefill");
    return prefill_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                        query_start_loc, max_query_len, scale, out, num_seqs, total_q,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                        PA_LAYOUT_TOKEN_MAJOR, stream);
}

pa_status_t pa_prefill_layout(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_tables, int max_blocks_per_seq,
                              const int32_t *context_lens, const int32_t *query_start_loc,
                              int max_query_len, float scale, void *out, int num_seqs,
                              int total_q, int num_q_heads, int num_kv_heads, int head_dim,
                              int block_size, int64_t num_blocks, pa_layout_t layout,
                              void *stream) {
    TraceRange r("pa_prefill_layout");
    return prefill_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                        query_start_loc, max_query_len, scale, out, num_seqs, total_q,
                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, layout,
                        stream);
}

pa_status_t pa_copy_blocks(void *const *caches, int num_caches, const int32_t *block_pairs,
                           int64_t num_pairs, int num_kv_heads, int head_dim, int block_size,
                           int64_t num_blocks, void *stream) {
    TraceRange r("pa_copy_blocks");
    if (num_pairs < 0) return PA_ERR_INVALID_ARG;
    const pa_status_t chk = check_pools(caches, num_caches, num_kv_heads, head_dim, block_size, num_blocks);
    if (chk != PA_OK) return chk;
    if (num_pairs == 0 || num_caches == 0) return PA_OK;
    if (!block_pairs || (reinterpret_cast<uintptr_t>(block_pairs) & 7u)) return PA_ERR_INVALID_ARG;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const cudaError_t e = pa::launch_copy_blocks(
        caches, num_caches, block_pairs, num_pairs, num_blocks,
        block_chunks_of(num_kv_heads, head_dim, block_size), sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_blocks_workspace_size(int num_rows, int64_t num_blocks) {
    if (num_rows < 0 || num_blocks <= 0 || num_blocks > INT32_MAX) return 0;
    return pa::blocks_workspace_bytes(num_rows, num_blocks);
}

pa_status_t pa_fork_blocks(void *const *caches, int num_caches, int32_t *block_tables,
                           int max_blocks_per_seq, int32_t *context_lens, int num_rows,
                           int32_t *ref_counts, const int32_t *parents, const int32_t *children,
                           int num_forks, int num_kv_heads, int head_dim, int block_size,
                           int64_t num_blocks, pa_layout_t layout, void *workspace,
                           size_t workspace_bytes, void *stream) {
    TraceRange r("pa_fork_blocks");
    if (num_forks < 0 || num_rows < 0 || max_blocks_per_seq < 0 || num_forks > num_rows)
        return PA_ERR_INVALID_ARG;
    if (layout != PA_LAYOUT_TOKEN_MAJOR && layout != PA_LAYOUT_HEAD_MAJOR) return PA_ERR_INVALID_ARG;
    pa_status_t chk = check_pools(caches, num_caches, num_kv_heads, head_dim, block_size, num_blocks);
    if (chk != PA_OK) return chk;
    if (num_forks == 0) return PA_OK;
    if (!block_tables || !context_lens || !ref_counts || !parents || !children ||
        max_blocks_per_seq == 0)
        return PA_ERR_INVALID_ARG;
    chk = check_workspace(workspace, workspace_bytes, num_rows, num_blocks);
    if (chk != PA_OK) return chk;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    pa::ForkArgs a{};
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.ref_counts = ref_counts;
    a.parents = parents;
    a.children = children;
    a.max_blocks = max_blocks_per_seq;
    a.num_rows = num_rows;
    a.num_forks = num_forks;
    a.block_size_log2 = log2_exact(block_size);
    a.num_kv_heads = num_kv_heads;
    a.head_major = layout == PA_LAYOUT_HEAD_MAJOR ? 1 : 0;
    a.block_chunks = block_chunks_of(num_kv_heads, head_dim, block_size);
    a.num_blocks = num_blocks;
    const cudaError_t e = pa::launch_fork_blocks(caches, num_caches, a, workspace, sms,
                                                 static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t pa_free_blocks(int32_t *block_tables, int max_blocks_per_seq, int32_t *context_lens,
                           int num_rows, int32_t *ref_counts, const int32_t *rows, int num_freed,
                           int block_size, int64_t num_blocks, void *stream) {
    TraceRange r("pa_free_blocks");
    if (num_freed < 0 || num_rows < 0 || max_blocks_per_seq < 0 || num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (!block_size_ok(block_size) || num_blocks > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (num_freed == 0) return PA_OK;
    if (!block_tables || !context_lens || !ref_counts || !rows || max_blocks_per_seq == 0)
        return PA_ERR_INVALID_ARG;
    const cudaError_t e = pa::launch_free_blocks(
        block_tables, max_blocks_per_seq, context_lens, num_rows, ref_counts, rows, num_freed,
        log2_exact(block_size), num_blocks, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t pa_compact_blocks(void *const *caches, int num_caches, int32_t *block_tables,
                              int max_blocks_per_seq, const int32_t *context_lens, int num_rows,
                              int32_t *ref_counts, int32_t *remap, int32_t *num_live,
                              int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                              void *workspace, size_t workspace_bytes, void *stream) {
    TraceRange r("pa_compact_blocks");
    if (num_rows < 0 || max_blocks_per_seq < 0) return PA_ERR_INVALID_ARG;
    pa_status_t chk = check_pools(caches, num_caches, num_kv_heads, head_dim, block_size, num_blocks);
    if (chk != PA_OK) return chk;
    if (!ref_counts || !remap || !num_live) return PA_ERR_INVALID_ARG;
    if (num_rows > 0 && (!block_tables || !context_lens || max_blocks_per_seq == 0))
        return PA_ERR_INVALID_ARG;
    chk = check_workspace(workspace, workspace_bytes, num_rows, num_blocks);
    if (chk != PA_OK) return chk;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    pa::CompactArgs a{};
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.ref_counts = ref_counts;
    a.remap = remap;
    a.num_live = num_live;
    a.max_blocks = max_blocks_per_seq;
    a.num_rows = num_rows;
    a.block_size_log2 = log2_exact(block_size);
    a.block_chunks = block_chunks_of(num_kv_heads, head_dim, block_size);
    a.num_blocks = num_blocks;
    const cudaError_t e = pa::launch_compact_blocks(caches, num_caches, a, workspace, sms,
                                                    static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_decode_tree_workspace_size(int num_q_heads, int num_kv_heads, int head_dim) {
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        head_dim != pa::kHeadDimPublic || pa::decode_group_pad(num_q_heads / num_kv_heads) == 0)
        return 0;
    const int sms = current_sm_count();
    return sms > 0 ? pa::tree_workspace_bytes(sms) : 0;
}

pa_status_t pa_decode_tree(const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, const int32_t *query_start_loc,
                           const uint64_t *tree_mask, int mask_words, float scale, void *out,
                           int num_seqs, int total_q, int num_q_heads, int num_kv_heads,
                           int head_dim, int block_size, int64_t num_blocks, pa_layout_t layout,
                           void *workspace, size_t workspace_bytes, void *stream) {
    TraceRange r("pa_decode_tree");
    if (total_q < 0 || mask_words < 1) return PA_ERR_INVALID_ARG;
    if (mask_words > PA_TREE_MAX_WORDS) return PA_ERR_UNSUPPORTED;
    bool nothing_to_do = false;
    const pa_status_t chk = pa::decode_check_args(
        q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, 1, scale, out,
        total_q > 0 ? num_seqs : 0, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, layout, 0,
        &nothing_to_do);
    if (chk != PA_OK) return chk;
    if (num_seqs < 0) return PA_ERR_INVALID_ARG;
    if ((int64_t)total_q * num_q_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX - 127) return PA_ERR_UNSUPPORTED;
    // the call counts places of all units in 32 bits
    if (!pa::tree_places_fit(total_q, pa::decode_group_pad(num_q_heads / num_kv_heads), num_seqs,
                             (int64_t)max_blocks_per_seq * block_size, num_kv_heads))
        return PA_ERR_UNSUPPORTED;
    if (nothing_to_do) return PA_OK;
    if (!query_start_loc || !tree_mask || (reinterpret_cast<uintptr_t>(tree_mask) & 7u)) return PA_ERR_INVALID_ARG;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    if (!workspace || !aligned16(workspace) || workspace_bytes < pa::tree_workspace_bytes(sms))
        return PA_ERR_WORKSPACE;
    pa::TreeArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.starts = query_start_loc;
    a.mask = reinterpret_cast<const uint32_t *>(tree_mask);
    a.out = out;
    a.mask_words = 2 * mask_words;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = num_q_heads / num_kv_heads;
    a.block_size_log2 = log2_exact(block_size);
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.head_major = layout == PA_LAYOUT_HEAD_MAJOR ? 1 : 0;
    a.box_tokens = block_size < 128 ? block_size : 128;
    a.fault_hold_v = pa::prefill_fault();
    a.num_blocks = num_blocks;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    // a scale of 0 stands for the smallest number: scores are then 0 to fp32, and a masked
    // one's infinity stays one
    if (a.scale_log2 == 0.f) a.scale_log2 = 1.4e-45f;
    a.workers = std::min(sms, pa::kTreeMaxWorkers);
    pa::tree_carve_workspace(a, workspace);
    const cudaError_t e = pa::launch_decode_tree(a, pa::decode_group_pad(a.group), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t pa_keep_tokens(void *const *caches, int num_caches, int32_t *block_tables,
                           int max_blocks_per_seq, int32_t *context_lens,
                           const int32_t *query_start_loc, const int32_t *kept, int max_kept,
                           int num_seqs, int32_t *ref_counts, int num_kv_heads, int head_dim,
                           int block_size, int64_t num_blocks, pa_layout_t layout, void *stream) {
    TraceRange r("pa_keep_tokens");
    if (num_seqs < 0 || max_blocks_per_seq < 0 || max_kept < 1) return PA_ERR_INVALID_ARG;
    if (layout != PA_LAYOUT_TOKEN_MAJOR && layout != PA_LAYOUT_HEAD_MAJOR) return PA_ERR_INVALID_ARG;
    const pa_status_t chk = check_pools(caches, num_caches, num_kv_heads, head_dim, block_size, num_blocks);
    if (chk != PA_OK) return chk;
    if (max_kept > PA_KEEP_MAX_TOKENS || num_seqs > 65535) return PA_ERR_UNSUPPORTED;
    if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!block_tables || !context_lens || !query_start_loc || !kept || max_blocks_per_seq == 0)
        return PA_ERR_INVALID_ARG;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    pa::KeepArgs a{};
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.starts = query_start_loc;
    a.kept = kept;
    a.ref_counts = ref_counts;
    a.max_blocks = max_blocks_per_seq;
    a.max_kept = max_kept;
    a.num_seqs = num_seqs;
    a.block_size_log2 = log2_exact(block_size);
    a.num_kv_heads = num_kv_heads;
    a.head_major = layout == PA_LAYOUT_HEAD_MAJOR ? 1 : 0;
    a.num_blocks = num_blocks;
    const cudaError_t e = pa::launch_keep_tokens(caches, num_caches, a, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t pa_rotary_init_frequencies(pa_rotary_t *rotary, int rot_dim, int interleaved,
                                       const double *frequencies, double amplitude) {
    if (!rotary || !frequencies || (interleaved != 0 && interleaved != 1)) return PA_ERR_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > 2 * PA_ROTARY_MAX_PAIRS || rot_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (!std::isfinite((float)amplitude)) return PA_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!(std::fabs(frequencies[i]) <= 1048576.0)) return PA_ERR_INVALID_ARG;
    pa::rotary_fill(rotary, rot_dim, interleaved, frequencies, amplitude);
    return PA_OK;
}

pa_status_t pa_rotary_init(pa_rotary_t *rotary, int rot_dim, int interleaved, double base,
                           pa_rotary_scaling_t scaling, double factor, double original_context,
                           double low, double high, double amplitude) {
    if (!(std::isfinite(base) && base > 1) || scaling < PA_ROTARY_PLAIN || scaling > PA_ROTARY_BANDED)
        return PA_ERR_INVALID_ARG;
    if (scaling != PA_ROTARY_PLAIN && !(std::isfinite(factor) && factor >= 1)) return PA_ERR_INVALID_ARG;
    if (scaling == PA_ROTARY_YARN || scaling == PA_ROTARY_BANDED) {
        if (!(std::isfinite(original_context) && original_context >= 1)) return PA_ERR_INVALID_ARG;
        if (!(low > 0 && std::isfinite(high) && low < high)) return PA_ERR_INVALID_ARG;
    }
    if (rot_dim < 16 || rot_dim > 2 * PA_ROTARY_MAX_PAIRS || rot_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    double radians[PA_ROTARY_MAX_PAIRS];
    pa::rotary_scaled(radians, rot_dim, base, scaling, factor, original_context, low, high);
    if (amplitude == 0) amplitude = scaling == PA_ROTARY_YARN ? 1 + 0.1 * std::log(factor) : 1;
    return pa_rotary_init_frequencies(rotary, rot_dim, interleaved, radians, amplitude);
}

pa_status_t pa_rotate(const void *q, int64_t q_token_stride, int64_t q_head_stride, void *q_out,
                      int64_t q_out_token_stride, int64_t q_out_head_stride, int num_q_heads,
                      const void *k, int64_t k_token_stride, int64_t k_head_stride, void *k_out,
                      int64_t k_out_token_stride, int64_t k_out_head_stride, int num_kv_heads,
                      int head_dim, const int32_t *positions, int64_t num_tokens,
                      const pa_rotary_t *rotary, const void *q_weight, const void *k_weight,
                      float eps, void *stream) {
    TraceRange r("pa_rotate");
    pa::RotateArgs a{};
    bool interleaved = false;
    const pa_status_t chk = rotate_args(a, &interleaved, q, q_token_stride, q_head_stride, q_out,
                                        q_out_token_stride, q_out_head_stride, num_q_heads, k,
                                        k_token_stride, k_head_stride, num_kv_heads, head_dim,
                                        positions, num_tokens, rotary, q_weight, k_weight, eps);
    if (chk != PA_OK) return chk;
    if (num_tokens == 0 || num_q_heads + num_kv_heads == 0) return PA_OK;
    if (num_kv_heads > 0 && (!rows_ok(k_out, num_tokens, k_out_token_stride, num_kv_heads, k_out_head_stride) ||
                             !rows_apart(num_tokens, k_out_token_stride, num_kv_heads, k_out_head_stride)))
        return PA_ERR_INVALID_ARG;
    a.k_out = {static_cast<uint4 *>(k_out), k_out_token_stride / 8, k_out_head_stride / 8};
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const cudaError_t e = pa::launch_rotate(a, false, interleaved, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t pa_append_kvcache(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                              void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                              int num_q_heads, const void *k, int64_t k_token_stride,
                              int64_t k_head_stride, const void *v, int64_t v_token_stride,
                              int64_t v_head_stride, int num_kv_heads, int head_dim, void *k_cache,
                              void *v_cache, const int64_t *slot_mapping, int block_size,
                              int64_t num_blocks, pa_layout_t layout, const int32_t *positions,
                              int64_t num_tokens, const pa_rotary_t *rotary, const void *q_weight,
                              const void *k_weight, float eps, void *stream) {
    TraceRange r("pa_append_kvcache");
    bool nothing_to_do = false;
    pa_status_t chk = pa::store_check_args(k, v, k_cache, v_cache, slot_mapping, num_tokens,
                                           num_kv_heads, head_dim, block_size, num_blocks, layout,
                                           &nothing_to_do);
    if (chk != PA_OK) return chk;
    pa::RotateArgs a{};
    bool interleaved = false;
    chk = rotate_args(a, &interleaved, q, q_token_stride, q_head_stride, q_out, q_out_token_stride,
                      q_out_head_stride, num_q_heads, k, k_token_stride, k_head_stride,
                      num_kv_heads, head_dim, positions, num_tokens, rotary, q_weight, k_weight, eps);
    if (chk != PA_OK || nothing_to_do) return chk;
    if (!rows_ok(v, num_tokens, v_token_stride, num_kv_heads, v_head_stride)) return PA_ERR_INVALID_ARG;
    a.v = {static_cast<const uint4 *>(v), v_token_stride / 8, v_head_stride / 8};
    a.k_cache = static_cast<uint4 *>(k_cache);
    a.v_cache = static_cast<uint4 *>(v_cache);
    a.slots = slot_mapping;
    a.num_slots = num_blocks * block_size;
    a.block_size_log2 = log2_exact(block_size);
    a.head_major = layout == PA_LAYOUT_HEAD_MAJOR ? 1 : 0;
    const int sms = current_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const cudaError_t e = pa::launch_rotate(a, true, interleaved, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status_t pa_debug_kernel_variant(int flags) {
    if (flags & ~(PA_VARIANT_DECODE_SIMT | PA_VARIANT_PREFILL_MMA)) return PA_ERR_INVALID_ARG;
    g_kernel_variant.store(flags, std::memory_order_relaxed);
    return PA_OK;
}

pa_status_t pa_debug_prefill_fault(int mode) {
    if (mode != 0 && mode != 1) return PA_ERR_INVALID_ARG;
    pa::set_prefill_fault(mode);
    return PA_OK;
}

pa_status_t pa_take_device_error(int32_t *code, void *stream) {
    TraceRange r("pa_take_device_error");
    if (!code) return PA_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t (*const take[])(cudaStream_t, int *) = {
        pa::take_prefill_error, pa::take_prefill_mma_error, pa::take_decode_error,
        pa::take_store_error,      pa::take_blocks_error,
        pa::take_shared_error, pa::take_rotary_error, pa::take_tree_error, pa::take_keep_error};
    int first = 0;
    for (auto f : take) {   // every word is read and cleared; the smallest code is reported
        int v = 0;
        if (f(st, &v) != cudaSuccess) return PA_ERR_CUDA;
        if (v != 0 && (first == 0 || v < first)) first = v;
    }
    *code = first;
    return PA_OK;
}

}  // extern "C"
