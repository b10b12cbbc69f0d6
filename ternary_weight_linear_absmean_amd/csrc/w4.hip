// w4.hip -- 4-bit weights with group scales: quantiser, its inverse, and the
// product with a few tokens.
//
// Per group of a row: a = max |w|, s = bf16(fl(a / 7)), code = clamp(rne(fl(w
// / s)), -7, 7); the quotients are correctly rounded, so codes and scales are
// defined to the bit.  A group is held by group / 8 neighbouring lanes, eight
// values each (one dword of codes), so its maximum is a few DPP steps and
// everything is read and written once.
#include "device_common.h"
#include "launch.h"

namespace bl {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t bf16_round(float x) {
    const uint32_t w = __float_as_uint(x);
    return (w + 0x7FFFu + (w >> 16 & 1u)) >> 16;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t at, float (&x)[8]) {
    if (BF16) {
        const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
        x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
        x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
    } else {
        const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        const float4 u = f[0], v = f[1];
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    }
}

__device__ __forceinline__ int w4_code(float x, float d) {
    const float r = __builtin_rintf(__fdiv_rn(x, d));
    return (int)fminf(fmaxf(r, -7.0f), 7.0f);
}

// n8 = N * K / 8 dwords of codes, in order: rows are whole groups, so a row's
// end never falls inside one.
template <bool BF16, int GROUP>
__global__ __launch_bounds__(kThreads) void quant_w4_kernel(const void *__restrict__ W, int64_t n8,
                                                            uint32_t *__restrict__ Wq4,
                                                            uint16_t *__restrict__ s4) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const bool in = i < n8;
    float x[8];
    load8<BF16>(W, 8 * (in ? i : n8 - 1), x);
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(x[j]));
    if (!in) a = 0.0f;
    a = group_max(a, GROUP / 8);
    const uint32_t sb = bf16_round(__fdiv_rn(a, 7.0f));
    const float d = __uint_as_float(sb << 16);
    uint32_t w = 0;
    if (d > 0.0f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w |= (uint32_t)(w4_code(x[j], d) & 15) << (4 * j);
    }
    if (in) {
        Wq4[i] = w;
        if (i % (GROUP / 8) == 0) s4[i / (GROUP / 8)] = (uint16_t)sb;
    }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void dequant_w4_kernel(const uint32_t *__restrict__ Wq4,
                                                              const uint16_t *__restrict__ s4,
                                                              int64_t n8, int g_shift,
                                                              void *__restrict__ W) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n8) return;
    const uint32_t w = Wq4[i];
    const float d = __uint_as_float((uint32_t)s4[i >> g_shift] << 16);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = (float)((int)(w << (28 - 4 * j)) >> 28) * d;
    if (BF16) {
        uint4 o;
        o.x = bf16_round(y[0]) | bf16_round(y[1]) << 16;
        o.y = bf16_round(y[2]) | bf16_round(y[3]) << 16;
        o.z = bf16_round(y[4]) | bf16_round(y[5]) << 16;
        o.w = bf16_round(y[6]) | bf16_round(y[7]) << 16;
        static_cast<uint4 *>(W)[i] = o;
    } else {
        float4 *o = static_cast<float4 *>(W) + 2 * i;
        o[0] = make_float4(y[0], y[1], y[2], y[3]);
        o[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
}

// One wave per (row of W, token).
template <bool BF16>
__global__ __launch_bounds__(kThreads) void gemv_w4_kernel(const void *__restrict__ X, int M,
                                                           const uint32_t *__restrict__ Wq4,
                                                           const uint16_t *__restrict__ s4, int N,
                                                           int K, int g_shift,
                                                           float *__restrict__ Y) {
    const int lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (i >= (int64_t)M * N) return;
    const int64_t n = i % N, m = i / N;
    float sum = 0.0f;
    for (int u = lane; u < K / 8; u += 64) {
        const int64_t at = n * (K / 8) + u;
        const uint32_t w = Wq4[at];
        const float d = __uint_as_float((uint32_t)s4[at >> g_shift] << 16);
        float x[8], y = 0.0f;
        load8<BF16>(X, m * K + 8 * u, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) y += x[j] * (float)((int)(w << (28 - 4 * j)) >> 28);
        sum += y * d;
    }
    for (int w = 1; w < 64; w <<= 1) sum += __shfl_xor(sum, w);
    if (lane == 0) Y[i] = sum;
}

int dword_shift(int group) { return group == 32 ? 2 : group == 64 ? 3 : 4; }

template <bool BF16>
void quant(const void *W, int64_t n8, int group, uint32_t *Wq4, uint16_t *s4, hipStream_t s) {
    const dim3 grid((unsigned)((n8 + kThreads - 1) / kThreads)), block(kThreads);
    if (group == 32)
        hipLaunchKernelGGL((quant_w4_kernel<BF16, 32>), grid, block, 0, s, W, n8, Wq4, s4);
    else if (group == 64)
        hipLaunchKernelGGL((quant_w4_kernel<BF16, 64>), grid, block, 0, s, W, n8, Wq4, s4);
    else
        hipLaunchKernelGGL((quant_w4_kernel<BF16, 128>), grid, block, 0, s, W, n8, Wq4, s4);
}

}  // namespace

hipError_t launch_quant_weight_i4(const void *W, int dtype, int64_t N, int64_t K, int group,
                                  uint8_t *Wq4, uint16_t *s4, hipStream_t s) {
    uint32_t *w = reinterpret_cast<uint32_t *>(Wq4);
    if (dtype)
        quant<true>(W, N * K / 8, group, w, s4, s);
    else
        quant<false>(W, N * K / 8, group, w, s4, s);
    return hipGetLastError();
}

hipError_t launch_dequant_weight_i4(const uint8_t *Wq4, const uint16_t *s4, int64_t N, int64_t K,
                                    int group, void *W, int dtype, hipStream_t s) {
    const int64_t n8 = N * K / 8;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(Wq4);
    const dim3 grid((unsigned)((n8 + kThreads - 1) / kThreads)), block(kThreads);
    if (dtype)
        hipLaunchKernelGGL(dequant_w4_kernel<true>, grid, block, 0, s, w, s4, n8,
                           dword_shift(group), W);
    else
        hipLaunchKernelGGL(dequant_w4_kernel<false>, grid, block, 0, s, w, s4, n8,
                           dword_shift(group), W);
    return hipGetLastError();
}

hipError_t launch_gemv_w4(const void *X, int dtype, int M, const uint8_t *Wq4, const uint16_t *s4,
                          int N, int K, int group, float *Y, hipStream_t s) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(Wq4);
    const dim3 grid((unsigned)(((int64_t)M * N + 3) / 4)), block(kThreads);
    if (dtype)
        hipLaunchKernelGGL(gemv_w4_kernel<true>, grid, block, 0, s, X, M, w, s4, N, K,
                           dword_shift(group), Y);
    else
        hipLaunchKernelGGL(gemv_w4_kernel<false>, grid, block, 0, s, X, M, w, s4, N, K,
                           dword_shift(group), Y);
    return hipGetLastError();
}

}  // namespace bl
