// kv_read.hip -- cached rows back as values, in the order of a call's rows.
//
// The value of a code is formed in fp32: fl(code s) for 8 bits, fl(z + code s)
// for 4 (code s is exact), then rounded to the rows' type.
//
// One workgroup per (16 consecutive positions of a sequence, HEADS heads), K and V,
// as the 4-bit append's groups.  K's codes are in the rows' order; V's are 16
// tokens of one value side by side and cross LDS.  A workgroup's time is its
// chain of loads (starts and length, table entry, codes), so where there are more of them
// than run at once each takes four heads, their loads all in flight.
//
// Bound by the values' bytes: 16 sequences of up to 4096 tokens, 5 heads of 128,
// bf16, from 4 bits, 170 MB: 30.2 us, 5.6 TB/s, a copy's rate.  64.7 us with K and V
// apart by head and stores through the caches, whose lines the end of a kernel
// writes out; 60.4 with four heads, 37.1 with stores past the caches, the rest K
// and V together.  500 tokens: 3.4 us, latency.
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
};

template <typename E, int D, int HEADS, typename C>
__global__ __launch_bounds__(2 * D) void kv_read_kernel(Args<C> a) {
    constexpr bool kFour = __is_same(C, Kv4Cache);
    constexpr int kPer = D / 8;                           // threads of a token
    __shared__ alignas(16) uint8_t codes[HEADS][16][D + 16];
    const Kv8Seqs &seqs = a.seqs;
    const C &c = a.c;
    const uint32_t chunks = (uint32_t)(c.KVH + HEADS - 1) / HEADS;
    const uint32_t slot = blockIdx.x / chunks;
    const int h0 = (int)(blockIdx.x - slot * chunks) * HEADS, heads = min(HEADS, c.KVH - h0);
    const SeqPlace in_seq = find_place(seqs, slot, [](int q, int i) { return (int64_t)(q >> 4) + 2 * (int64_t)i; });
    const int b = in_seq.b, q0 = in_seq.q0, n = in_seq.q1 - q0;
    const int64_t nth = (int64_t)slot - ((q0 >> 4) + 2 * (int64_t)b);
    if (nth < 0 || n <= 0) return;
    const int64_t len = in_seq.length, start = len - n;
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
    const int64_t to = ((q0 + (pos - start)) * c.KVH + h0) * (int64_t)D + 8 * td;
    E *const k = static_cast<E *>(a.k) + to, *const v = static_cast<E *>(a.v) + to;
    if (!held) {
        if (mine)
            for (int i = 0; i < heads; ++i) {
                const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
                store_row4(k + i * D, none);
                store_row4(k + i * D + 4, none);
                store_row4(v + i * D, none);
                store_row4(v + i * D + 4, none);
            }
        return;
    }
    const int64_t head = (int64_t)id * c.KVH + h0;
    const int in = (int)(16 * j & (c.T - 1));             // first of the 16 slots
    uint32_t sk[HEADS], sv[HEADS];                        // z and s, or a scale
    uint2 u[HEADS];                                       // this thread's codes of K
    uint4 g[HEADS];                                       // value threadIdx.x of the 16 tokens of V
    const int vd = min((int)threadIdx.x, D - 1);
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int64_t hi = head + min(i, heads - 1);
        if constexpr (kFour) {
            sk[i] = c.zk[hi * c.T + in + t];
            sv[i] = c.zv[hi * c.T + in + t];
            u[i].x = *reinterpret_cast<const uint32_t *>(c.K + (hi * c.T + in + t) * (int64_t)(D / 2) + 4 * td);
            const uint2 w = *reinterpret_cast<const uint2 *>(c.V + (hi * (c.T / 16) + in / 16) * (int64_t)(8 * D) + 8 * vd);
            g[i].x = w.x;
            g[i].y = w.y;
        } else {
            sk[i] = __float_as_uint(c.sk[hi]);
            sv[i] = __float_as_uint(c.sv[hi]);
            u[i] = *reinterpret_cast<const uint2 *>(c.K + (hi * c.T + in + t) * (int64_t)D + 8 * td);
            g[i] = *reinterpret_cast<const uint4 *>(c.V + (hi * D + vd) * (int64_t)c.T + in);
        }
    }
    auto put = [&](E *to, uint32_t scale, uint2 p, int shift) {      // 8 codes, a byte or 4 bits of it each
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t x = (e < 4 ? p.x : p.y) >> (8 * (e & 3));
            if constexpr (kFour) w[e] = __builtin_fmaf((float)(x >> shift & 15u), (float)zs_s(scale), (float)zs_z(scale));
            else w[e] = __fmul_rn((float)(int8_t)x, __uint_as_float(scale));
        }
        store_row4(to, make_float4(w[0], w[1], w[2], w[3]));
        store_row4(to + 4, make_float4(w[4], w[5], w[6], w[7]));
    };
    if (threadIdx.x < D) {
        // line of LDS: a token, or two of 4 bits
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
            const uint32_t w[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
            for (int y = 0; y < (kFour ? 8 : 16); ++y) codes[i][y][threadIdx.x] = (uint8_t)(w[y >> 2] >> (8 * (y & 3)));
        }
    }
    if (mine) {
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
            if (i >= heads) break;
            uint2 p = u[i];
            if constexpr (kFour) {                        // values 2 e, 2 e + 1 of byte e -> bytes
                const uint32_t lo = u[i].x & 0x0F0F0F0Fu, hi = u[i].x >> 4 & 0x0F0F0F0Fu;
                p = make_uint2(perm(hi, lo, 0x05010400u), perm(hi, lo, 0x07030602u));
            }
            put(k + i * D, sk[i], p, 0);
        }
    }
    __syncthreads();
    if (!mine) return;
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        if (i >= heads) break;
        put(v + i * D, sv[i], *reinterpret_cast<const uint2 *>(&codes[i][kFour ? t >> 1 : t][8 * td]), kFour ? 4 * (t & 1) : 0);
    }
}

// A call of four times the threads that run at once takes four heads a workgroup
// (of 0.6 times, 4355 tokens of 8 heads of 64: 8.7 us by head, 9.5 by four, K and V
// apart).
constexpr int64_t kAtOnce = 4 * 256 * 2048;

template <typename E, int D, typename C>
hipError_t read(const Kv8Seqs &seqs, const C &c, void *k, void *v, hipStream_t s) {
    const Args<C> a = {seqs, c, k, v};
    static_assert(sizeof a <= kFewArgs, "a launch's arguments");
    const int64_t slots = (seqs.n_tok >> 4) + 2 * (int64_t)seqs.B;
    const bool four = slots * c.KVH * 2 * D > kAtOnce;
    const int64_t groups = slots * (four ? (c.KVH + 3) / 4 : c.KVH);
    if (groups * 2 * D >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
    if (four)
        hipLaunchKernelGGL((kv_read_kernel<E, D, 4, C>), dim3((unsigned)groups), dim3(2 * D), 0, s, a);
    else
        hipLaunchKernelGGL((kv_read_kernel<E, D, 1, C>), dim3((unsigned)groups), dim3(2 * D), 0, s, a);
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
