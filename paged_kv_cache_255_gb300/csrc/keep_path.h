// The list of kept nodes of a draft: which of its entries continue the path. Plain C++, so
// that the CPU can go through lists of every kind.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PA_PATH_FN __host__ __device__ __forceinline__
#else
#define PA_PATH_FN inline
#endif

namespace pa {

// Whether entry i of a list continues the path that the entries before it are, k and `before`
// being entries i and i - 1 (`before` is not looked at for i = 0), n the draft's nodes; `bad`
// when it ends the list and is no -1.
//
// The path ends at the first entry that does not continue it; what stands behind that one is
// nobody's, and a thread that looks at an entry alone does not know whether it is behind.
// So an entry that continues names the places i and k of the draft, 0 <= i <= k < n, wherever
// it stands: a path ascends from 0 or above, so that its entry i is at least i.
PA_PATH_FN bool path_continues(int k, int before, int i, int n, bool &bad) {
    const bool ok = k >= i && k < n && (i == 0 || k > before);
    bad = !ok && k != -1;
    return ok;
}

}  // namespace pa
