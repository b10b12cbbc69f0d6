// kv4_common.h -- the 4-bit key/value cache as the kernels take it.
#pragma once

#include "kv_common.h"

namespace bl {

// K [block][head][T][D / 2] and V [block][head][T / 16][D][8] in bytes of two
// codes; zk, zv [block][head][T]: a token's least value z (fp16) in the lower
// half, its step s (fp16) in the upper.
struct Kv4Cache {
    uint8_t *K, *V;
    uint32_t *zk, *zv;
    int n_blocks, KVH, T, D;
    int t_shift;                  // log2(T)
};

inline void *scales1(const Kv4Cache &c) { return c.zk; }
inline void *scales2(const Kv4Cache &c) { return c.zv; }
template <>
__device__ __forceinline__ Kv4Cache cache_of<Kv4Cache>(void *K, void *V, void *s1, void *s2, int n_blocks, int KVH,
                                                     int t_shift, int D) {
    return {static_cast<uint8_t *>(K), static_cast<uint8_t *>(V), static_cast<uint32_t *>(s1), static_cast<uint32_t *>(s2), n_blocks, KVH,
            1 << t_shift, D, t_shift};
}

inline Kv4Cache kv4_device(const bl_kv4 &c) {
    Kv4Cache d = {c.K, c.V, reinterpret_cast<uint32_t *>(c.zk), reinterpret_cast<uint32_t *>(c.zv),
                  (int)c.n_blocks, (int)c.KVH, (int)c.T, (int)c.D, 0};
    while ((1 << d.t_shift) < d.T) ++d.t_shift;
    return d;
}

// Halves of a z, s pair.
__device__ __forceinline__ _Float16 zs_z(uint32_t w) { return __builtin_bit_cast(half2, w)[0]; }
__device__ __forceinline__ _Float16 zs_s(uint32_t w) { return __builtin_bit_cast(half2, w)[1]; }

}  // namespace bl
