// Where the parts of an output row of decode over shared prefixes are: the
// checks of the records that the kernels before the combine leave, and the slots
// that an accepted record leads to. Plain C++, so that the CPU can go through
// all records.
//
// A share that gave up waiting for its tiles leaves no record, and the workspace
// then holds whatever was there: a record of an earlier call, of another kind
// of unit, or no record at all. The launch's outputs are undefined in that case;
// what is read must still lie in the workspace.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PA_RECORD_FN __host__ __device__ __forceinline__
#else
#define PA_RECORD_FN inline
#endif

namespace pa {

constexpr int kRecordWhole = -1;    // the unit's rows are whole, in whole_o
constexpr int kRecordDone = -2;     // nothing is left of it: its share has written the output

// A record {first slot or one of the above, last share, first share} of a unit
// of decode_shared_kernel, which has 2 slots for each of `workers` shares. An own part
// may be done; a packed prefix never is.
template <class R>
PA_RECORD_FN bool unit_record_ok(const R &r, int workers, bool may_be_done) {
    return r.x >= (may_be_done ? kRecordDone : kRecordWhole) && r.x < 2 * workers && r.z >= 0 && r.z <= r.y &&
           r.y < workers && (r.x < 0 || r.x >> 1 == r.z);
}

// A record {first slot, parts, slots between them} of a unit of the prefix
// kernel, which has 2 slots for each of `workers` CTAs; all 0 where there is no
// such unit.
template <class R>
PA_RECORD_FN bool prefix_record_ok(const R &r, int workers) {
    return r.x >= 0 && r.y >= 0 && r.y <= workers && r.z >= 0 && r.z <= 2 * workers &&
           (r.x | 1) + (int64_t)(r.y - 1) * r.z < 2 * workers;
}

// The slot of part `at`: a share's first piece is where its record says, the
// next shares' at their even slots, `apart` slots from one to the next.
PA_RECORD_FN int64_t record_slot(int first, int at, int apart) {
    return (int64_t)(at == 0 ? first : (first & ~1) + at * apart);
}

}  // namespace pa
