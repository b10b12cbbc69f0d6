// kv_common.h -- what the calls on the paged key/value caches share: the arrays
// of a call's sequences.
#pragma once

#include "device_common.h"
#include "launch.h"

namespace bl {

// q_start[b] taken within the call's rows.
__device__ __forceinline__ int q_at(const Kv8Seqs &s, int b) {
    return min(max(s.q_start[b], 0), s.n_tok);
}

// The largest b in [0, B) with first(b) <= i, first non-decreasing; 0 when
// there is none.  A wave looks at 64 entries at a time, so up to 64 sequences
// take one load and up to 4096 two.  With entries that decrease the result is
// some b in [0, B).  Every lane of the wave must be active; i is uniform.
template <typename F>
__device__ __forceinline__ int find_seq(int B, int64_t i, F first) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = B;
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int at = lane * step;
        const bool below = at < n && first(lo + at) <= i;
        const int c = max(__popcll(__ballot(below)), 1) - 1;
        lo += c * step;
        n = min(step, n - c * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

}  // namespace bl
