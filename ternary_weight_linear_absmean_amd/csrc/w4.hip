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

// ---------------------------------------------------------------------------
// Y [M][N] = X W^T, M <= 16.  Two kernels: fp32 multiply-adds for one or two
// tokens, fp16 matrix instructions from three on.
//
// A 4-bit code is exact in fp16: with its sign bit flipped it is code + 8;
// below the byte 0x64 that reads as 1024 + (code + 8) from bits 0..3 and as
// 1024 + 16 (code + 8) from bits 4..7, and one packed add or multiply-add
// leaves the code: 10 instructions per dword of 8 codes, in the order 0, 4, 1,
// 5, 2, 6, 3, 7.
//
// In both, the waves of a workgroup share its rows of W and divide K among
// them, so that a wave's part of X stays in its registers for all the rows,
// W is read with 16-byte loads that are all in flight together, and nothing
// but the final sums (in the waves' order) goes through LDS.
struct Codes {
    half2 p[4];               // codes 0, 4 | 1, 5 | 2, 6 | 3, 7
};
__device__ __forceinline__ Codes codes_to_f16(uint32_t w) {
    const uint32_t x = w ^ 0x88888888u, y = x >> 8;
    const half2 low = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const half2 mul = {(_Float16)0.0625f, (_Float16)0.0625f}, high = {(_Float16)-72.0f, (_Float16)-72.0f};
    auto h = [](uint32_t v) { return __builtin_bit_cast(half2, v); };
    Codes c;
    c.p[0] = h((x & 0x000F000Fu) | 0x64006400u) + low;
    c.p[1] = __builtin_elementwise_fma(h((x & 0x00F000F0u) | 0x64006400u), mul, high);
    c.p[2] = h((y & 0x000F000Fu) | 0x64006400u) + low;
    c.p[3] = __builtin_elementwise_fma(h((y & 0x00F000F0u) | 0x64006400u), mul, high);
    return c;
}

struct ProdArgs {
    const void *X;
    const uint32_t *Wq4;
    const uint16_t *s4;
    float *Y;
    int M, N, K;
};

constexpr int kMaxWaves = 8;

// One or two tokens.  A wave takes slices of 512 values of K: 16 lanes hold 32
// values each of X in fp32 and the same 32 codes of a row (16 bytes, within
// one scale group), four rows at a time, R times.
constexpr int kSlice = 512;
template <bool BF16, int M, int R>
__global__ __launch_bounds__(64 * kMaxWaves) void gemv_w4_few_kernel(ProdArgs a, int g_shift) {
    __shared__ float red[kMaxWaves][M][4 * R];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int kl = lane & 15, rg = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (4 * R);
    const int units = a.K / 32, groups = units >> g_shift;      // 16-byte units and scales of a row
    float acc[M][R];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[m][r] = 0.0f;
    for (int u0 = wave * 16; u0 < units; u0 += waves * 16) {
        const bool in = u0 + kl < units;
        const int u = in ? u0 + kl : units - 1;
        uint4 w[R];
        uint16_t sb[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t n = min(n0 + 4 * r + rg, (int64_t)a.N - 1);
            w[r] = reinterpret_cast<const uint4 *>(a.Wq4)[n * units + u];
            sb[r] = a.s4[n * groups + (u >> g_shift)];
        }
        float x[M][4][8];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) load8<BF16>(a.X, (int64_t)m * a.K + 32 * u + 8 * j, x[m][j]);
        if (!in) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[m][j][e] = 0.0f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t ww[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
            float s0[M], s1[M];
#pragma unroll
            for (int m = 0; m < M; ++m) s0[m] = s1[m] = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Codes c = codes_to_f16(ww[j]);
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s0[m] = __builtin_fmaf((float)c.p[e][0], x[m][j][e], s0[m]);
                        s1[m] = __builtin_fmaf((float)c.p[e][1], x[m][j][e + 4], s1[m]);
                    }
            }
            const float d = __uint_as_float((uint32_t)sb[r] << 16);
#pragma unroll
            for (int m = 0; m < M; ++m) acc[m][r] = __builtin_fmaf(s0[m] + s1[m], d, acc[m][r]);
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v = acc[m][r];
            v += dpp_f32<kDppXor1>(v);
            v += dpp_f32<kDppXor2>(v);
            v += dpp_f32<kDppHalfMirror>(v);
            v += dpp_f32<kDppMirror>(v);
            if (kl == 0) red[wave][m][4 * r + rg] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < M * 4 * R; i += blockDim.x) {
        const int m = i / (4 * R), n = i % (4 * R);
        float y = red[0][m][n];
        for (int v = 1; v < waves; ++v) y += red[v][m][n];
        if (n0 + n < a.N) a.Y[m * (int64_t)a.N + n0 + n] = y;
    }
}

// Three tokens and more: 16x16x32 products, A = 16 tokens x 32 values of X, B =
// 32 values x 16 rows of W.  A wave takes chunks of 128 values; lane 16 quad +
// low holds 32 values of token `low`, and 16 bytes of row `low` per 16 rows of
// W, R times.
//
// X is scaled by a power of two per token and chunk, the largest to [2^13,
// 2^14), and rounded to fp16: bf16 values are exact (down to 2^-31 of the
// largest), fp32 values are split in two halves of 11 bits, each with its
// matrix instructions.
//
// A matrix instruction sums over the four quads, and all that it sums has to
// lie in one scale group.  With groups of 128 any dword of each quad's 16 bytes
// will do; with 32 the quads have to bring the four dwords of one lane, which
// is a transpose of the 4 x 4 dwords between registers and quads (4 row swaps
// per 16 bytes); with 64 half of it.  X is loaded in the order this makes.  The
// sum of a group leaves the matrix accumulators once, times X's factor and the
// scale, into fp32 totals.
constexpr int kChunk = 128;

__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

template <bool BF16, int GROUP, int R>
__global__ __launch_bounds__(64 * kMaxWaves) void gemv_w4_mfma_kernel(ProdArgs a) {
    constexpr int NS = BF16 ? 1 : 2;
    constexpr int NG = kChunk / GROUP;          // groups of a chunk
    __shared__ float red[kMaxWaves][R][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int low = lane & 15, quad = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * R);
    const int units = a.K / 32, groups = a.K / GROUP;
    const int64_t xrow = (int64_t)min(low, a.M - 1) * a.K;
    float4v tot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) tot[r] = float4v{0.f, 0.f, 0.f, 0.f};

    for (int c = wave; c * kChunk < a.K; c += waves) {
        // K is a multiple of 32, so a chunk's end falls between units
        uint4 w[R];
        uint16_t sb[R][NG];
        const int u = c * 4 + quad;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t n = min(n0 + 16 * r + low, (int64_t)a.N - 1);
            w[r] = reinterpret_cast<const uint4 *>(a.Wq4)[n * units + min(u, units - 1)];
#pragma unroll
            for (int g = 0; g < NG; ++g) sb[r][g] = a.s4[n * groups + min(c * NG + g, groups - 1)];
        }
        float x[4][8];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // the 8 values that matrix instruction j takes from this quad:
            // dword dj of quad dq's 16 bytes
            const int dq = GROUP == 128 ? quad : GROUP == 64 ? (quad & 1) | (j & 2) : j;
            const int dj = GROUP == 128 ? j : GROUP == 64 ? (j & 1) | (quad & 2) : quad;
            const int uu = c * 4 + dq;
            load8<BF16>(a.X, xrow + 32 * (int64_t)min(uu, units - 1) + 8 * dj, x[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (uu >= units) x[j][e] = 0.0f;
                top = fmaxf(top, fabsf(x[j][e]));
            }
        }
        top = quad_max(top);
        // top in [2^(e-127), 2^(e-126)) -> [2^13, 2^14), in two factors as
        // their product may pass fp32's range
        const int ex = max((int)(__float_as_uint(top) >> 23), 1);
        const int e1 = (140 - ex) / 2, e2 = 140 - ex - e1;
        const float f1 = __uint_as_float((uint32_t)(127 + e1) << 23);
        const float f2 = __uint_as_float((uint32_t)(127 + e2) << 23);
        // 2^(ex - 140), exact (as a subnormal where ex < 14)
        const float back = __uint_as_float((uint32_t)(127 - e1) << 23) *
                           __uint_as_float((uint32_t)(127 - e2) << 23);
        half8 xh[NS][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h[4], z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {                  // in the codes' order
                const float v0 = x[j][e] * f1 * f2, v1 = x[j][e + 4] * f1 * f2;
                h[e] = f16_pair(v0, v1);
                if (NS == 2) z[e] = f16_rest(v0, v1, h[e]);
            }
            xh[0][j] = __builtin_bit_cast(half8, make_uint4(h[0], h[1], h[2], h[3]));
            if (NS == 2) xh[NS - 1][j] = __builtin_bit_cast(half8, make_uint4(z[0], z[1], z[2], z[3]));
        }
        // the factors of the tokens whose sums this lane gets
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __shfl(back, 4 * quad + e);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t d[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
            if (NG >= 2) {
                swap32(d[0], d[2]);
                swap32(d[1], d[3]);
            }
            if (NG == 4) {
                swap16(d[0], d[1]);
                swap16(d[2], d[3]);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float4v acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = g * (4 / NG); j < (g + 1) * (4 / NG); ++j) {
                    const half8 b = __builtin_bit_cast(half8, codes_to_f16(d[j]));
#pragma unroll
                    for (int s = 0; s < NS; ++s) acc = mfma_16x16x32(xh[s][j], b, acc);
                }
                const float sc = __uint_as_float((uint32_t)sb[r][g] << 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) tot[r][e] = __builtin_fmaf(acc[e] * f[e], sc, tot[r][e]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[wave][r][e][lane] = tot[r][e];
    __syncthreads();
    for (int i = threadIdx.x; i < R * 256; i += blockDim.x) {
        const int r = i >> 8, e = i >> 6 & 3, l = i & 63;
        const int m = 4 * (l >> 4) + e;
        const int64_t n = n0 + 16 * r + (l & 15);
        if (m >= a.M || n >= a.N) continue;
        float y = red[0][r][e][l];
        for (int v = 1; v < waves; ++v) y += red[v][r][e][l];
        a.Y[m * (int64_t)a.N + n] = y;
    }
}

// Waves for `parts` of K: as few as keep the longest share of a wave.
int waves_for(int parts) {
    if (parts <= kMaxWaves) return parts > 0 ? parts : 1;
    const int share = (parts + kMaxWaves - 1) / kMaxWaves;
    return (parts + share - 1) / share;
}

template <bool BF16, int M, int R>
void few(const ProdArgs &a, int group, hipStream_t s) {
    const unsigned grid = (unsigned)((a.N + 4 * R - 1) / (4 * R));
    const int waves = waves_for((a.K + kSlice - 1) / kSlice);
    hipLaunchKernelGGL((gemv_w4_few_kernel<BF16, M, R>), dim3(grid), dim3(64 * waves), 0, s, a,
                       group == 32 ? 0 : group == 64 ? 1 : 2);
}
template <bool BF16, int GROUP, int R>
void many(const ProdArgs &a, hipStream_t s) {
    const unsigned grid = (unsigned)((a.N + 16 * R - 1) / (16 * R));
    const int waves = waves_for((a.K + kChunk - 1) / kChunk);
    hipLaunchKernelGGL((gemv_w4_mfma_kernel<BF16, GROUP, R>), dim3(grid), dim3(64 * waves), 0, s, a);
}
template <bool BF16, int GROUP>
void many(const ProdArgs &a, hipStream_t s) {
    if (a.N >= 16384) many<BF16, GROUP, 4>(a, s);
    else many<BF16, GROUP, 1>(a, s);
}

template <bool BF16>
void product(const ProdArgs &a, int group, hipStream_t s) {
    if (a.M == 1) {
        if (a.N >= 8192) few<BF16, 1, 8>(a, group, s);
        else few<BF16, 1, 2>(a, group, s);
    } else if (a.M == 2) {
        if (a.N >= 8192) few<BF16, 2, 8>(a, group, s);
        else few<BF16, 2, 2>(a, group, s);
    } else if (group == 32) {
        many<BF16, 32>(a, s);
    } else if (group == 64) {
        many<BF16, 64>(a, s);
    } else {
        many<BF16, 128>(a, s);
    }
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
    ProdArgs a = {X, reinterpret_cast<const uint32_t *>(Wq4), s4, Y, M, N, K};
    if (dtype)
        product<true>(a, group, s);
    else
        product<false>(a, group, s);
    return hipGetLastError();
}

}  // namespace bl
