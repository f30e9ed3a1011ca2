// How the heads of a rotation are shared among warps. Plain C++, so that the CPU can go through
// sizes of every kind.
#pragma once

#include <cstdint>

namespace pa {

struct RotarySplit {
    int quads;      // groups of four heads a warp takes of a token
    int slices;     // warps a token's heads are shared among
};

// A warp takes as many of a token's quads as leave the GPU full of warps: the sines are then
// computed once for all of them. (One wave of 24 warps an SM, each going from token to
// token, instead of CTAs in turn: 16384 tokens of 40 heads 58.9 us against 52.5, of 2047 x 48
// 19.1 against 14.5.)
//
// Several slices a token are few tokens: with places = 32 sm_count, more than one means
// num_tokens < places, and then num_tokens * slices < 3 places. So items, num_tokens * slices,
// are below 2^31 for any size and are counted in 32 bits.
inline RotarySplit rotary_split(int64_t num_tokens, int rows, int sm_count) {
    const int all = (rows + 3) / 4;
    const int64_t fill = num_tokens * all / ((int64_t)sm_count * 32);
    const int most = (int)(fill < 1 ? 1 : (fill > all ? all : fill));
    const int slices = (all + most - 1) / most;
    return RotarySplit{(all + slices - 1) / slices, slices};    // alike
}

}  // namespace pa
