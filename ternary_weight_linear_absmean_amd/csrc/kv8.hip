// kv8.hip -- new key / value rows into the 8-bit cache.
//
// Per block and head, for K and for V apart: a = max |x| over the new rows of
// the block, d = fl(a / 127), not below the scale of the block's earlier
// tokens; where the scale grows, the block's codes become rne(fl(code *
// fl(s / d))); new codes are clamp(rne(fl(x / d)), -127, 127).  Quotients are
// correctly rounded, so the cache's bytes are defined to the bit.
//
// One workgroup per (touched block, head, K or V): it alone writes that
// block, so nothing is shared between workgroups and no order of them
// matters.  The grid is known without the lengths: sequence b with n_b new
// tokens touches at most ceil(n_b / T) + 1 blocks, and the slots
//     first(b) = floor(q_start[b] / T) + 2 b
// leave it floor(q_start[b+1] / T) - floor(q_start[b] / T) + 2 of them, which
// is never fewer; floor(n_tok / T) + 2 B slots in all.  Unused ones exit.
//
// Decode is bound by latency: starts, length, table entry, rows, maximum and
// quotient follow one another (64 sequences, 5 heads of 128: 6.1 us, 2 of them
// the launch).  Prompts are one pass over the rows, held in registers between
// the maximum and the codes (4400 fp32 rows, 27 MB: 10.9 us, 2.5 TB/s, start and
// end of one wave of workgroups; a multiplication with a check in the place of
// the correctly rounded quotients took 5% off).
#include "kv8_common.h"

namespace bl {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4(const uint16_t *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

__device__ __forceinline__ int kv8_code(float x, float d) {
    const float r = __builtin_rintf(__fdiv_rn(x, d));
    return (int)fminf(fmaxf(r, -127.0f), 127.0f);
}
__device__ __forceinline__ uint32_t kv8_code4(float4 x, float d) {
    if (!(d > 0.0f)) return 0u;
    return (uint32_t)(kv8_code(x.x, d) & 255) | (uint32_t)(kv8_code(x.y, d) & 255) << 8 |
           (uint32_t)(kv8_code(x.z, d) & 255) << 16 | (uint32_t)(kv8_code(x.w, d) & 255) << 24;
}
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float r) {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = (float)(int)(int8_t)(w >> (8 * i));
        o |= (uint32_t)((int)__builtin_rintf(__fmul_rn(c, r)) & 255) << (8 * i);
    }
    return o;
}

// NC = T * D / (4 * kThreads): 4-value pieces of a whole block per thread.
template <typename E, int NC>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(const E *__restrict__ k,
                                                              const E *__restrict__ v,
                                                              Kv8Seqs seqs, Kv8Cache c) {
    __shared__ alignas(16) uint32_t tile[NC * kThreads];   // the new codes, [slot][D]
    __shared__ float wave_max[kThreads / 64];
    const int T = c.T, D = c.D, sh = c.t_shift;
    const int64_t slot = blockIdx.x;
    const int h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;

    const int b = find_seq(seqs.B, slot, [&](int i) {
        return (int64_t)(q_at(seqs, i) >> sh) + 2 * (int64_t)i;
    });
    const int q0 = q_at(seqs, b);
    const int64_t nth = slot - ((q0 >> sh) + 2 * (int64_t)b);
    const int n = q_at(seqs, b + 1) - q0;
    if (nth < 0 || n <= 0) return;
    const int64_t len = seqs.lengths[b];
    const int64_t start = len - n;                     // position of row q0
    const int64_t j = (max(start, (int64_t)0) >> sh) + nth;
    if (j >= seqs.max_blocks) return;
    const int64_t first = max(max(start, (int64_t)0), j << sh);
    const int64_t last = min(len, (j + 1) << sh);
    if (first >= last) return;
    const int id = seqs.table[(int64_t)b * seqs.max_blocks + j];
    const int s0 = (int)(first - (j << sh)), s1 = (int)(last - (j << sh));   // the new slots
    const int units = D / 4;                           // per row
    const int total = (s1 - s0) * units;
    const E *x = (is_v ? v : k) + ((q0 + (first - start)) * c.KVH + h) * (int64_t)D;
    const int64_t row_step = (int64_t)c.KVH * D;
    const int u_shift = D == 64 ? 4 : 5;

    // the new rows of this block and head, all loads in flight together (at
    // clamped addresses: a branch around each would serialise them)
    float4 r[NC];
    float a = 0.0f;
    const int pieces = total <= kThreads ? 1 : NC;
    if (pieces == 1) {
        const int u = min((int)threadIdx.x, total - 1);
        r[0] = load4(x + (u >> u_shift) * row_step + 4 * (u & (units - 1)));
        a = fmaxf(fmaxf(fabsf(r[0].x), fabsf(r[0].y)), fmaxf(fabsf(r[0].z), fabsf(r[0].w)));
    } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int u = min((int)threadIdx.x + i * kThreads, total - 1);
            r[i] = load4(x + (u >> u_shift) * row_step + 4 * (u & (units - 1)));
        }
#pragma unroll
        for (int i = 0; i < NC; ++i)
            a = fmaxf(a, fmaxf(fmaxf(fabsf(r[i].x), fabsf(r[i].y)),
                               fmaxf(fabsf(r[i].z), fabsf(r[i].w))));
    }
    if (id < 0 || id >= c.n_blocks) return;            // uniform: the block holds no token
    const int64_t hb = (int64_t)id * c.KVH + h;
    float *scale = (is_v ? c.sv : c.sk) + hb;
    const float before = s0 > 0 ? *scale : 0.0f;       // s0 > 0: earlier tokens in the block

    a = group_max(a, 64);
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = a;
    __syncthreads();
    a = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
    const float fresh = __fdiv_rn(a, 127.0f);
    const float d = s0 > 0 ? fmaxf(before, fresh) : fresh;
    const bool grown = s0 > 0 && d > before;
    const float fit = grown ? __fdiv_rn(before, d) : 1.0f;
    if (threadIdx.x == 0) *scale = d;

#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int u = (int)threadIdx.x + i * kThreads;
        if (i < pieces && u < total) tile[u] = kv8_code4(r[i], d);
    }
    __syncthreads();

    const int8_t *codes = reinterpret_cast<const int8_t *>(tile);    // row 0 = slot s0
    int8_t *dst = (is_v ? c.V : c.K) + hb * (int64_t)(T * D);
    for (int u = threadIdx.x; u < T * D / 16; u += kThreads) {
        if (!is_v) {
            const int at = u * 16;                      // [slot][D]
            const int s = at / D;
            uint4 *p = reinterpret_cast<uint4 *>(dst + at);
            if (s >= s0 && s < s1) {
                *p = *reinterpret_cast<const uint4 *>(codes + at - s0 * D);
            } else if (grown) {
                uint4 w = *p;
                w.x = rescale_codes(w.x, fit);
                w.y = rescale_codes(w.y, fit);
                w.z = rescale_codes(w.z, fit);
                w.w = rescale_codes(w.w, fit);
                *p = w;
            }
        } else {
            // [D][slot]: 16 slots of one value; lanes take neighbouring values
            const int dd = u & (D - 1), t0 = (u >> (D == 64 ? 6 : 7)) * 16;
            int8_t *p8 = dst + dd * T + t0;
            const int lo = max(s0, t0), hi = min(s1, t0 + 16);
            if (!grown) {
                if (lo == t0 && hi == t0 + 16) {
                    uint4 w;
                    uint32_t *ww = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t o = 0;
#pragma unroll
                        for (int jj = 0; jj < 4; ++jj)
                            o |= (uint32_t)(uint8_t)codes[(t0 - s0 + 4 * i + jj) * D + dd] << (8 * jj);
                        ww[i] = o;
                    }
                    *reinterpret_cast<uint4 *>(p8) = w;
                } else {
                    for (int s = lo; s < hi; ++s) p8[s - t0] = codes[(s - s0) * D + dd];
                }
            } else {
                uint4 w = *reinterpret_cast<const uint4 *>(p8);
                w.x = rescale_codes(w.x, fit);
                w.y = rescale_codes(w.y, fit);
                w.z = rescale_codes(w.z, fit);
                w.w = rescale_codes(w.w, fit);
                uint32_t *ww = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int s = t0 + i;
                    if (s >= s0 && s < s1) {
                        const uint32_t m = 255u << (8 * (i & 3));
                        ww[i >> 2] = (ww[i >> 2] & ~m) |
                                     (uint32_t)(uint8_t)codes[(s - s0) * D + dd] << (8 * (i & 3));
                    }
                }
                *reinterpret_cast<uint4 *>(p8) = w;
            }
        }
    }
}

template <typename E>
hipError_t append(const E *k, const E *v, const Kv8Seqs &seqs, const Kv8Cache &c, hipStream_t s) {
    const int64_t slots = (seqs.n_tok >> c.t_shift) + 2 * (int64_t)seqs.B;
    const dim3 grid((unsigned)slots, (unsigned)c.KVH, 2), block(kThreads);
    switch (c.T * c.D / (4 * kThreads)) {
    case 1: hipLaunchKernelGGL((kv8_append_kernel<E, 1>), grid, block, 0, s, k, v, seqs, c); break;
    case 2: hipLaunchKernelGGL((kv8_append_kernel<E, 2>), grid, block, 0, s, k, v, seqs, c); break;
    case 4: hipLaunchKernelGGL((kv8_append_kernel<E, 4>), grid, block, 0, s, k, v, seqs, c); break;
    case 8: hipLaunchKernelGGL((kv8_append_kernel<E, 8>), grid, block, 0, s, k, v, seqs, c); break;
    default: hipLaunchKernelGGL((kv8_append_kernel<E, 16>), grid, block, 0, s, k, v, seqs, c);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv8_append(const void *k, const void *v, int dtype, const Kv8Seqs &seqs,
                             const bl_kv8 &cache, hipStream_t s) {
    const Kv8Cache c = kv8_device(cache);
    return dtype ? append(static_cast<const uint16_t *>(k), static_cast<const uint16_t *>(v), seqs,
                          c, s)
                 : append(static_cast<const float *>(k), static_cast<const float *>(v), seqs, c, s);
}

}  // namespace bl
