// How decode over trees counts its work: what of a batch is a sequence's, and the places of
// its units in the flat space that is shared among the CTAs. Plain C++, so that the CPU can go
// through starts and lengths of every kind.
#pragma once

#include <climits>
#include <cstdint>

#ifdef __CUDACC__
#define PA_TREE_FN __host__ __device__ __forceinline__
#else
#define PA_TREE_FN inline
#endif

namespace pa {

constexpr int kTreePairRows = 256;      // query rows of a unit
constexpr int kTreeKeys = 128;          // keys of a tile
// Places of a unit besides its tiles, for its start and its end (measured in tree.cu).
constexpr int kTreeUnitPlaces = 3;

// A sequence's part of the work.
struct TreeSeq {
    int q0, n, L;       // first query row, query rows (nodes; negative where the starts fall), tokens
    int nt, pairs;      // key tiles; units of 256 query rows
};

// Of starts q0, q1 and length l as the caller's arrays hold them; G rows a token, max_len
// (below 2^31) the tokens of a table.
PA_TREE_FN TreeSeq tree_seq(int q0, int q1, int l, int total_q, int64_t max_len, int G) {
    q0 = q0 < 0 ? 0 : (q0 > total_q ? total_q : q0);
    q1 = q1 < 0 ? 0 : (q1 > total_q ? total_q : q1);
    TreeSeq r;
    r.q0 = q0;
    r.n = q1 - q0;
    r.L = (int)(l < 0 ? 0 : (l > max_len ? max_len : l));
    r.nt = r.L > 0 ? (r.L + kTreeKeys - 1) / kTreeKeys : 1;     // an empty sequence's zeros are written by one tile
    r.pairs = r.n > 0 ? (int)(((int64_t)r.n * G + kTreePairRows - 1) / kTreePairRows) : 0;
    return r;
}

// Places of a sequence's units, below 2^31 where tree_places_fit.
PA_TREE_FN int tree_seq_places(const TreeSeq &q, int num_kv_heads) {
    return q.pairs * num_kv_heads * (q.nt + kTreeUnitPlaces);
}

// Lanes that units are shared in: where all sequences with units have the same number of
// them a KV head, these go side by side and read the same keys together, each lane over
// workers / lanes CTAs, as long as the CTAs left over, workers modulo lanes, are an eighth at
// most. Otherwise there is one lane, whose shares take every CTA. Of 152 CTAs, us side by side
// and in one lane: 8 units a KV head over 100000 tokens, 8 heads, 545 and 591; 13 (9 CTAs left
// over) 942 and 1066; 17 (16) 645 and 740; one head over 16000 tokens 22 (20) 48.9 and 48.4,
// 32 (24) 67 and 64, 52 (48) 125 and 99, 77 (75) 231 and 143.
PA_TREE_FN int tree_lanes(int most, int least, int workers) {
    return most > 1 && most == least && most <= workers && workers % most <= workers / 8 ? most : 1;
}

// Whether the places of all sequences of a call, whatever its lengths, are below 2^31, as
// long as no start is below the one before it: the rows of two sequences are then not the
// same, and there are total_q of them in all. The kernel counts again where one is.
inline bool tree_places_fit(int total_q, int G, int num_seqs, int64_t max_len, int num_kv_heads) {
    const int64_t units = (int64_t)total_q * G / kTreePairRows + num_seqs;
    const int64_t tiles = (max_len + kTreeKeys - 1) / kTreeKeys + 8;
    return tiles * num_kv_heads <= INT32_MAX && units <= INT32_MAX / (tiles * num_kv_heads);
}

}  // namespace pa
