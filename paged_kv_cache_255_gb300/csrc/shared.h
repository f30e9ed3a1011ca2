// Plan, buffers and launches of decode over shared prefixes (shared.cu plans
// and computes the prefixes, decode.cu the rest of every sequence).
#pragma once

#include <atomic>

#include "kernels.h"

namespace pa {

constexpr int kSharedMaxGroups = 4096;  // groups of one call (the plan keeps 20 bytes each in shared memory)
constexpr int kSharedMinSeqs = 2;       // a prefix is computed apart for at least this many sequences
// What a unit of decode_shared_kernel costs besides its tiles (its queries, its
// result), in tiles. Without it the shares of many short units ended up to 9 us
// after the others (60 sequences of 1 .. 500 own tokens).
constexpr int kUnitTiles = 4;
// Sequences whose heads fit the 8 columns of one unit of decode_shared_kernel: a
// power of two.
__host__ __device__ constexpr int shared_fit_log2(int group) {
    return group == 1 ? 3 : group == 2 ? 2 : group <= 4 ? 1 : 0;
}
__host__ __device__ constexpr int shared_fit(int group) { return 1 << shared_fit_log2(group); }
constexpr int kPairRows = 256;      // rows of a prefix unit: two query tiles of 128

// A group whose prefix is computed once. Its tile space: (KV head, pair of
// query tiles, key tile), the key tile fastest, from `base` on.
struct alignas(16) SharedGroup {
    int base;           // flat index of the group's first key tile
    int unit;           // index of its first unit in SharedArgs::parts
    int row;            // table row the prefix is read through
    int s0, n;          // its sequences
    int tokens;         // prefix tokens computed together, a multiple of 16
    int nt, pairs;      // key tiles of 128; pairs of query tiles
};
static_assert(sizeof(SharedGroup) == 32, "one 32-byte sector");

// A share's walk over the tile space: its pieces are runs of key tiles
// [j0, j1) of one unit, a unit being 256 query rows of one (group, KV head). Where
// all groups have the same number of pairs, the pairs are lanes: a share stays in one
// lane, the lanes are cut alike, and T counts the tiles of a lane. Otherwise there
// is one lane, of all pairs.
struct alignas(16) SharedWalk {
    int64_t T, T1;          // next tile, end of the share
    SharedGroup gr;
    int act, kvh, pair, j0, j1;
    int lane, lanes;
};

struct SharedHeader {
    int64_t tiles;          // prefix: key tiles of a lane
    int64_t own_tiles;      // decode.cu: 16-token tiles of all units, and kUnitTiles for each
    int s_lo, s_hi;         // sequences the call covers
    int entries;            // of SharedArgs::entries
    int workers;            // CTAs the prefix tiles are shared among
    int lanes, shares;      // worker w has share w / lanes of lane w % lanes, of `shares`
    int own_workers;        // warps the own tiles are shared among
};

// An entry of decode_shared_kernel's work list: for every KV head, a unit of
// the tokens [start, len) of a table row for `cols` query rows.
struct alignas(16) SharedUnit {
    int row;                // table row
    int first;              // sequence of the first query row; the heads of the next ones follow
    int start, len;         // start is a multiple of 16
    int cols;
    int part;               // other parts of the same query rows exist: +1; it is a prefix: +2
    int pad[2];
};

// Pointers are device memory.
struct SharedArgs {
    const int32_t *group_starts;    // [num_groups + 1]
    const int32_t *prefix_blocks;   // [num_groups]
    int num_groups;
    int group_pad;                  // G: query heads per KV head, rounded up to a power of two
    int max_workers;                // CTAs of the prefix kernel
    int box_tokens;                 // tokens of a TMA box of the prefix kernel: min(block size, 128)
    int tensor;                     // whether the prefix kernel is launched
    int fault_hold_v;               // test hook, normally 0: see set_prefill_fault
    // in the workspace
    SharedHeader *hdr;
    int4 *seq;                      // [S] {unit of KV head 0 or -1, entry of its packed prefix or -1,
                                    //      row of the unit or column of the entry, units of a KV head}
    SharedUnit *entries;            // [2 S] own tokens of every covered sequence, then packed prefixes
    long long *scan;                // [2 S] the same of one KV head, through an entry
    SharedGroup *groups;            // [num_groups] the active ones
    SharedWalk *walks;              // [max_workers] first piece of every share
    int4 *parts;                    // [S Hkv] a prefix unit's {first slot, parts, slots between them};
                                    // slot 2 w is worker w's first piece, 2 w + 1 its last
    float4 *part_o;                 // [2 max_workers][32][256] pieces of units that several workers share
    float2 *part_ml;                // [2 max_workers][256] (running max in log2 units, sum)
    float4 *unit_o;                 // [Hkv][32][S G] units one worker computed whole
    float2 *unit_ml;                // [Hkv][S G]
    int4 *units;                    // [2 S Hkv] where the parts of an entry's units are (decode.cu)
    float4 *whole_o;                // [2 S Hq][32] units one share computed whole: own, then packed
    float2 *whole_ml;               // [2 S Hq]
};

// Raises a kernel's limit of dynamic shared memory, once on every device.
class SmemLimit {
  public:
    cudaError_t raise(const void *kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = (uint64_t)1 << (dev & 63);     // the library's calls take devices 0 .. 63
        if (done_.load(std::memory_order_relaxed) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }

  private:
    std::atomic<uint64_t> done_{0};
};

size_t shared_workspace_bytes(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads,
                              int group_pad, int sm_count);
void shared_carve_workspace(SharedArgs &sh, void *workspace, const DecodeArgs &a);

// Plan and prefixes, then (launch_decode_shared) the rest and the combine.
cudaError_t launch_shared_prefix(const DecodeArgs &a, const SharedArgs &sh, cudaStream_t stream);
cudaError_t launch_decode_shared(const DecodeArgs &a, const SharedArgs &sh, cudaStream_t stream);
cudaError_t take_shared_error(cudaStream_t stream, int *code);

}  // namespace pa
