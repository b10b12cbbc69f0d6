// kv_read.hip -- cached rows back as values, in the order of a call's rows.
//
// The value of a code is formed in fp32: fl(code s) for 8 bits, fl(z + code s)
// for 4 (code s is exact), then rounded to the rows' type.
//
// One workgroup per (16 consecutive positions of a sequence, head, K or V), as
// the 4-bit append's.  K's codes are in the rows' order; V's are 16 tokens of
// one value side by side and cross LDS.
#include "kv4_common.h"
#include "kv8_common.h"
#include "rope.h"

namespace bl {
namespace {

template <typename C>
struct Args {
    Kv8Seqs seqs;
    C c;
    void *k, *v;
    int64_t slots;
};

template <typename E, int D, typename C>
__global__ __launch_bounds__(2 * D) void kv_read_kernel(Args<C> a) {
    constexpr bool kFour = __is_same(C, Kv4Cache);
    constexpr int kPer = D / 8;                           // threads of a token
    __shared__ alignas(16) uint8_t codes[16][D + 16];
    const Kv8Seqs &seqs = a.seqs;
    const C &c = a.c;
    const uint32_t pair = blockIdx.x / 2, slot = pair / (uint32_t)c.KVH;
    const bool is_v = blockIdx.x & 1;
    const int h = (int)(pair - slot * c.KVH);
    const int b = find_seq(seqs.B, slot, [&](int i) { return (int64_t)(q_at(seqs, i) >> 4) + 2 * (int64_t)i; });
    const int q0 = q_at(seqs, b), n = q_at(seqs, b + 1) - q0;
    const int64_t nth = (int64_t)slot - ((q0 >> 4) + 2 * (int64_t)b);
    if (nth < 0 || n <= 0) return;
    const int64_t len = seqs.lengths[b], start = len - n;
    const int64_t j = (start >> 4) + nth;                 // below 0 for positions that hold no token
    const int64_t first = max(start, 16 * j), last = min(len, 16 * j + 16);
    if (first >= last) return;
    int id = -1;
    if (j >= 0 && j < (int64_t)seqs.max_blocks << c.t_shift >> 4)
        id = seqs.table[(int64_t)b * seqs.max_blocks + (16 * j >> c.t_shift)];
    const bool held = id >= 0 && id < c.n_blocks;         // uniform
    const int t = threadIdx.x / kPer, td = threadIdx.x % kPer;
    const int64_t pos = 16 * j + t;
    const bool mine = pos >= first && pos < last;
    float4 o[2] = {};
    if (held) {
        const int64_t head = (int64_t)id * c.KVH + h;
        const int in = (int)(16 * j & (c.T - 1));         // first of the 16 slots
        float w[8];
        if constexpr (kFour) {
            const uint32_t zs = (is_v ? c.zv : c.zk)[head * c.T + in + t];
            uint32_t u = 0;
            if (!is_v) {
                u = *reinterpret_cast<const uint32_t *>(c.K + (head * c.T + in + t) * (int64_t)(D / 2) + 4 * td);
            } else {
                // value d's 8 bytes, two tokens to a byte; line i of LDS: tokens 2i, 2i + 1
                if (threadIdx.x < D) {
                    const uint2 g = *reinterpret_cast<const uint2 *>(
                        c.V + (head * (c.T / 16) + in / 16) * (int64_t)(8 * D) + 8 * threadIdx.x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        codes[i][threadIdx.x] = (uint8_t)(g.x >> (8 * i));
                        codes[4 + i][threadIdx.x] = (uint8_t)(g.y >> (8 * i));
                    }
                }
                __syncthreads();
                const uint2 p = *reinterpret_cast<const uint2 *>(&codes[t >> 1][8 * td]);
                const int sh = 4 * (t & 1);
                const uint32_t x = p.x >> sh & 0x0F0F0F0Fu, y = p.y >> sh & 0x0F0F0F0Fu;
#pragma unroll
                for (int e = 0; e < 4; ++e) u |= (x >> (8 * e) & 15u) << (4 * e) | (y >> (8 * e) & 15u) << (16 + 4 * e);
            }
            const float z = (float)zs_z(zs), s = (float)zs_s(zs);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __builtin_fmaf((float)(u >> (4 * e) & 15u), s, z);
        } else {
            const float s = (is_v ? c.sv : c.sk)[head];
            uint2 u;
            if (!is_v) {
                u = *reinterpret_cast<const uint2 *>(c.K + (head * c.T + in + t) * (int64_t)D + 8 * td);
            } else {
                if (threadIdx.x < D) {
                    const uint4 g = *reinterpret_cast<const uint4 *>(c.V + (head * D + threadIdx.x) * (int64_t)c.T + in);
                    const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                    for (int i = 0; i < 16; ++i) codes[i][threadIdx.x] = (uint8_t)(gw[i >> 2] >> (8 * (i & 3)));
                }
                __syncthreads();
                u = *reinterpret_cast<const uint2 *>(&codes[t][8 * td]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = __fmul_rn((float)(int8_t)(u.x >> (8 * e)), s);
                w[4 + e] = __fmul_rn((float)(int8_t)(u.y >> (8 * e)), s);
            }
        }
        o[0] = make_float4(w[0], w[1], w[2], w[3]);
        o[1] = make_float4(w[4], w[5], w[6], w[7]);
    }
    if (!mine) return;
    E *dst = static_cast<E *>(is_v ? a.v : a.k) + ((q0 + (pos - start)) * c.KVH + h) * (int64_t)D + 8 * td;
    store_row4(dst, o[0]);
    store_row4(dst + 4, o[1]);
}

template <typename E, int D, typename C>
hipError_t read(const Kv8Seqs &seqs, const C &c, void *k, void *v, hipStream_t s) {
    const Args<C> a = {seqs, c, k, v, (seqs.n_tok >> 4) + 2 * (int64_t)seqs.B};
    const int64_t groups = a.slots * c.KVH * 2;
    if (groups * 2 * D >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((kv_read_kernel<E, D, C>), dim3((unsigned)groups), dim3(2 * D), 0, s, a);
    return hipGetLastError();
}
template <typename C>
hipError_t read(const Kv8Seqs &seqs, const C &c, void *k, void *v, int dtype, hipStream_t s) {
    if (c.D == 64) return dtype ? read<uint16_t, 64>(seqs, c, k, v, s) : read<float, 64>(seqs, c, k, v, s);
    return dtype ? read<uint16_t, 128>(seqs, c, k, v, s) : read<float, 128>(seqs, c, k, v, s);
}

}  // namespace

hipError_t launch_kv8_read(const Kv8Seqs &seqs, const bl_kv8 &cache, void *k, void *v, int dtype, hipStream_t s) {
    return read(seqs, kv8_device(cache), k, v, dtype, s);
}
hipError_t launch_kv4_read(const Kv8Seqs &seqs, const bl_kv4 &cache, void *k, void *v, int dtype, hipStream_t s) {
    return read(seqs, kv4_device(cache), k, v, dtype, s);
}

}  // namespace bl
