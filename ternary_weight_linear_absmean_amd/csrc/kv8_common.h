// kv8_common.h -- the 8-bit key/value cache as the kernels take it.
#pragma once

#include "kv_common.h"

namespace bl {

// One block of the cache in bytes, and the tokens and values it is made of.
struct Kv8Cache {
    int8_t *K, *V;
    float *sk, *sv;
    int n_blocks, KVH, T, D;
    int t_shift;                  // log2(T)
};

inline void *scales1(const Kv8Cache &c) { return c.sk; }
inline void *scales2(const Kv8Cache &c) { return c.sv; }
template <>
__device__ __forceinline__ Kv8Cache cache_of<Kv8Cache>(void *K, void *V, void *s1, void *s2, int n_blocks, int KVH,
                                                     int t_shift, int D) {
    return {static_cast<int8_t *>(K), static_cast<int8_t *>(V), static_cast<float *>(s1), static_cast<float *>(s2), n_blocks, KVH,
            1 << t_shift, D, t_shift};
}

inline Kv8Cache kv8_device(const bl_kv8 &c) {
    Kv8Cache d = {c.K, c.V, c.sk, c.sv, (int)c.n_blocks, (int)c.KVH, (int)c.T, (int)c.D, 0};
    while ((1 << d.t_shift) < d.T) ++d.t_shift;
    return d;
}

}  // namespace bl
