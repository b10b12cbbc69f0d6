// kv_common.h -- what the calls on the paged key/value caches share: the arrays
// of a call's sequences.
#pragma once

#include "device_common.h"
#include "launch.h"

namespace bl {

// Bytes of a kernel's arguments up to which a launch takes the host 2.8 us; with a
// few more it is 3.3 to 4.0 (as the hidden ones that blockDim and gridDim bring with them).
constexpr size_t kFewArgs = 112;

// A cache's device view of its parts (kv8_common.h, kv4_common.h).
template <class C>
__device__ __forceinline__ C cache_of(void *K, void *V, void *s1, void *s2, int n_blocks, int KVH, int t_shift, int D);

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

// find_seq with what a kernel asks of the sequence next, its rows and length; first
// takes q_start[b] and b.  Up to 64 sequences take one step of loads in all (a
// wait for each after another costs a decode step 0.5 us).
struct SeqPlace {
    int b, q0, q1, length;
};
template <typename F>
__device__ __forceinline__ SeqPlace find_place(const Kv8Seqs &s, int64_t i, F first) {
    if (s.B <= 64) {
        const int lane = threadIdx.x & 63, at = min(lane, s.B - 1);
        const int q = q_at(s, at), next = q_at(s, at + 1), length = s.lengths[at];
        const uint64_t below = __ballot(lane < s.B && first(q, lane) <= i);
        const int b = max(__popcll(below), 1) - 1;
        return {b, __builtin_amdgcn_readlane(q, b), __builtin_amdgcn_readlane(next, b),
                __builtin_amdgcn_readlane(length, b)};
    }
    const int b = find_seq(s.B, i, [&](int at) { return (int64_t)first(q_at(s, at), at); });
    return {b, q_at(s, b), q_at(s, b + 1), s.lengths[b]};
}

}  // namespace bl
