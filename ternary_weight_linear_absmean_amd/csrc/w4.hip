// w4.hip -- 4-bit weights with group scales: quantiser, its inverse, and the
// product with a few tokens.
//
// Per group of a row: a = max |w|, s = bf16(fl(a / 7)), code = clamp(rne(fl(w
// / s)), -7, 7); the quotients are correctly rounded, so codes and scales are
// defined to the bit.  A group is held by group / 8 neighbouring lanes, eight
// values each (one dword of codes), so its maximum is a few DPP steps and
// everything is read and written once.  Both directions are bound by memory:
// 6912 x 2560 fp32 (80 MB) 13.6 us to codes and 15.4 us back, 5.2 to 5.9 TB/s
// with part of the matrix in the last cache.
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
// Y [M][N] = X W^T, M <= 16, in three forms: one or two tokens in fp32
// multiply-adds, with X in registers or, for many rows, in LDS; from three tokens
// on matrix instructions, fp16 for fp32 tokens and bf16 for bf16 tokens.
//
// A 4-bit code is exact in fp16: with its sign bit flipped it is code + 8;
// below the byte 0x64 that reads as 1024 + (code + 8) from bits 0..3 and as
// 1024 + 16 (code + 8) from bits 4..7, and one packed add or multiply-add
// leaves the code: 10 instructions per dword of 8 codes, in the order 0, 4, 1,
// 5, 2, 6, 3, 7.
//
// In the first and the last form the waves of a workgroup share its rows of W
// and divide K among them, so that a wave's part of X serves all the rows, W is
// read with 16-byte loads that are all in flight together, and the sums are
// joined once, in the waves' order, through LDS.
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

constexpr int kCUs = 256;
constexpr int kMaxWaves = 8;

// One or two tokens.  A wave takes slices of 512 values of K: 16 lanes hold 32
// values each of X in fp32 and the same 32 codes of a row (16 bytes, within
// one scale group), four rows at a time, R times.  Products and sums are fp32
// multiply-adds with a half of a register as the one factor.  2560 x 2560: 3.9
// us, launch and one round trip to memory (3.4 MB: 0.7 us).
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

// One or two tokens and many rows: X in LDS (fp32), every wave for itself.  A
// wave takes 4 R rows at a time through all of K (> 0), one slice's X in registers
// for its R loads, the next slice's loads in flight.  128256 x 2560 fp32 tokens,
// 174 MB: 42.6 us, 4.1 TB/s.
//
// X costs the other kernel a reading for every 16 rows, and this one a start, so
// this one is taken from 32768 rows on, with fp32 tokens from 16384 / M (measured
// at K = 2560 alone; both the start and a row's work grow with K): N x 2560, the
// other kernel and this one in us, M = 1: 12288 fp32 7.5 8.2, 24576 13.0 10.8,
// bf16 10.6 11.0, 40000 17.2 15.1; M = 2: 8192 fp32 9.1 8.5, 20000 18.8 13.3, bf16
// 13.0 13.4.  R = 2 for fewer than 65536 rows, of which a wave then has two tiles
// at most (40000: 15.1, 17.2 with 4), 4 from there on (98304: 34.0, 31.8).
constexpr int kStreamThreads = 256;
constexpr int kStreamGroups = 1024;
constexpr size_t kStreamLds = 64 * 1024;
constexpr int kStreamRows = 32768, kWideRows = 65536;
size_t stream_lds(int M, int K) {
    return (size_t)M * ((K + kSlice - 1) / kSlice) * kSlice * sizeof(float);
}
template <bool BF16, int M, int R>
__global__ __launch_bounds__(kStreamThreads, 4) void gemv_w4_stream_kernel(ProdArgs a, int g_shift) {
    extern __shared__ float xs[];               // [M][slices][8][16][4]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int kl = lane & 15, rg = lane >> 4;
    const int units = a.K / 32, groups = units >> g_shift;
    const int slices = (units + 15) / 16;
    // 16 bytes e of the 128 of lane kl stand at [slice][e][kl]: a read of one
    // e by 16 lanes is 256 consecutive bytes
    for (int i = threadIdx.x; i < M * slices * 64; i += kStreamThreads) {
        const int m = i / (slices * 64), k = (i - m * slices * 64) * 8;
        float x[8];
        load8<BF16>(a.X, (int64_t)m * a.K + min(k, a.K - 8), x);
        if (k >= a.K) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.0f;
        }
        const int sl = k / kSlice, l = k / 32 % 16, e = k / 8 % 4;
        float *d = xs + (((m * slices + sl) * 8 + 2 * e) * 16 + l) * 4;
        *reinterpret_cast<float4 *>(d) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(d + 64) = make_float4(x[4], x[5], x[6], x[7]);
    }
    __syncthreads();
    const int tiles = (int)(((uint32_t)a.N + 4 * R - 1) / (4 * R));
    const int step = gridDim.x * (kStreamThreads / 64);
    int tile = blockIdx.x * (kStreamThreads / 64) + wave;
    uint4 w[R];
    uint32_t sb[R];
    auto load_w = [&](int t, int sl) {
        const int u = min(sl * 16 + kl, units - 1);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t n = min((int64_t)t * (4 * R) + 4 * r + rg, (int64_t)a.N - 1);
            w[r] = reinterpret_cast<const uint4 *>(a.Wq4)[n * units + u];
            sb[r] = a.s4[n * groups + (u >> g_shift)];
        }
    };
    if (tile < tiles) load_w(tile, 0);
    for (; tile < tiles; tile += step) {
        float acc[M][R];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[m][r] = 0.0f;
        for (int sl = 0; sl < slices; ++sl) {
            uint4 wc[R];
            float d[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                wc[r] = w[r];
                d[r] = __uint_as_float(sb[r] << 16);
            }
            const bool end = sl + 1 == slices;
            load_w(end ? min(tile + step, tiles - 1) : tile, end ? 0 : sl + 1);
            float4 x[M][8];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[m][e] = *reinterpret_cast<const float4 *>(xs + (((m * slices + sl) * 8 + e) * 16 + kl) * 4);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t ww[4] = {wc[r].x, wc[r].y, wc[r].z, wc[r].w};
                float s0[M], s1[M];
#pragma unroll
                for (int m = 0; m < M; ++m) s0[m] = s1[m] = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Codes c = codes_to_f16(ww[j]);
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const float4 lo = x[m][2 * j], hi = x[m][2 * j + 1];
                        s0[m] = __builtin_fmaf((float)c.p[0][0], lo.x, s0[m]);
                        s1[m] = __builtin_fmaf((float)c.p[0][1], hi.x, s1[m]);
                        s0[m] = __builtin_fmaf((float)c.p[1][0], lo.y, s0[m]);
                        s1[m] = __builtin_fmaf((float)c.p[1][1], hi.y, s1[m]);
                        s0[m] = __builtin_fmaf((float)c.p[2][0], lo.z, s0[m]);
                        s1[m] = __builtin_fmaf((float)c.p[2][1], hi.z, s1[m]);
                        s0[m] = __builtin_fmaf((float)c.p[3][0], lo.w, s0[m]);
                        s1[m] = __builtin_fmaf((float)c.p[3][1], hi.w, s1[m]);
                    }
                }
#pragma unroll
                for (int m = 0; m < M; ++m)
                    acc[m][r] = __builtin_fmaf(s0[m] + s1[m], d[r], acc[m][r]);
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
                const int64_t n = (int64_t)tile * (4 * R) + 4 * r + rg;
                if (kl == 0 && n < a.N) a.Y[m * (int64_t)a.N + n] = v;
            }
    }
}

// Three tokens and more: 16x16x32 products, A = 16 tokens x 32 values of X, B =
// 32 values x 16 rows of W.  A wave takes chunks of 128 values: 16 bytes of row
// `low` per 16 rows of W, R times, and the tokens' values, loaded in whole
// lines (16 lanes a token), made fp16 and passed through LDS of the wave's own
// into the operand's order.
//
// bf16 tokens go into bf16 products as they are, in the codes' order, with the
// codes + 24: exact, and one instruction for two codes beside a shift (codes + 8
// by way of fp32, two conversions and a packing for two codes: 9.8 us where this
// takes 7.1, 16 x 6912 in groups of 32).  A product of the same X with -24 goes
// before each of them, so that the sums stay small; for the first of a group it is
// the same for all rows of W.  The numbers grow by a factor of about 6 for it,
// against the 2^-24 of the fp32 sums (all of a group's -24 first: by 12, and 2%
// faster with groups of 128).
//
// fp32 tokens are scaled by a power of two per token and chunk, the largest to
// [2^13, 2^14), and split in two fp16 halves of 11 bits, each with its matrix
// instructions.
//
// A matrix instruction sums over the four quads, and all that it sums has to
// lie in one scale group.  With groups of 128 any dword of each quad's 16 bytes
// will do; with 32 the quads have to bring the four dwords of one lane, which
// is a transpose of the 4 x 4 dwords between registers and quads (4 row swaps
// per 16 bytes); with 64 half of it.  place() is where 8 values of X belong
// then.  The sum of a group leaves the matrix accumulators once, times X's
// factor and the scale, into fp32 totals.
//
// 16 x 6912 -> 2560 bf16: 7.1 us, 11.4 MB; 160 workgroups of 16 rows, each with
// all of X (221 KB) through its registers: latency and vector instructions in
// equal parts.  More workgroups would read X oftener or need a join.
constexpr int kChunk = 128;

// Matrix instruction (dword) and quad that the 8 values of dword j of quad sq's
// 16 bytes go to: 4 instruction + quad.
template <int GROUP>
__device__ __forceinline__ int place(int sq, int j) {
    if (GROUP == 128) return j << 2 | sq;
    if (GROUP == 64) return ((j & 1) | (sq & 2)) << 2 | ((sq & 1) | (j & 2));
    return sq << 2 | j;
}

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

// Between a wave's writes and reads of LDS by different lanes (the hardware
// keeps their order; the compiler has to).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
__device__ __forceinline__ float4v mfma_bf16(bf8v a, bf8v b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// The 8 codes of a dword, + 24, as bf16 in the order 0, 4, 1, 5, 2, 6, 3, 7: with
// its sign bit flipped a code is code + 8, and below the bits of 16 that reads as
// 16 + (code + 8).
__device__ __forceinline__ bf8v codes_to_bf16(uint32_t w) {
    const uint32_t mask = 0x00780078u, base = 0x41C041C0u;       // 16, and the sign bit to flip
    return __builtin_bit_cast(bf8v, make_uint4(((w << 3) & mask) ^ base, ((w >> 1) & mask) ^ base,
                                               ((w >> 5) & mask) ^ base, ((w >> 9) & mask) ^ base));
}

// LDS of a wave: [part of X][instruction, quad][16 tokens + 1 of padding] units
// of 16 bytes, then 16 factors; the final sums take its place.
template <bool BF16>
constexpr int wave_lds() { return (BF16 ? 1 : 2) * 16 * 17 * 16 + 64; }

// WHOLE: K % 128 == 0 and s aligned to the scales of a chunk.
template <bool BF16, int GROUP, int R, bool WHOLE, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void gemv_w4_mfma_kernel(ProdArgs a) {
    constexpr int NS = BF16 ? 1 : 2;
    constexpr int NG = kChunk / GROUP;          // groups of a chunk
    extern __shared__ uint4 lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int low = lane & 15, quad = lane >> 4;
    uint4 *xs = lds + wave * (wave_lds<BF16>() / 16);
    float *xf = reinterpret_cast<float *>(xs + NS * 16 * 17);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * R);
    const int units = a.K / 32, groups = a.K / GROUP, chunks = (units + 3) / 4;
    float4v tot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) tot[r] = float4v{0.f, 0.f, 0.f, 0.f};

    for (int c = wave; c < chunks; c += waves) {
        // K is a multiple of 32, so its end falls between units; codes behind
        // it count 0, whatever X they meet (the row's last)
        uint4 w[R];
        float sc[R][NG];
        const int u = c * 4 + quad;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t n = min(n0 + 16 * r + low, (int64_t)a.N - 1);
            w[r] = reinterpret_cast<const uint4 *>(a.Wq4)[n * units + (WHOLE ? u : min(u, units - 1))];
            const uint16_t *sp = a.s4 + n * groups + c * NG;
            if (WHOLE && NG == 4) {
                const uint2 v = *reinterpret_cast<const uint2 *>(sp);
                sc[r][0] = bf16_lo(v.x);
                sc[r][1 % NG] = bf16_hi(v.x);
                sc[r][2 % NG] = bf16_lo(v.y);
                sc[r][3 % NG] = bf16_hi(v.y);
            } else if (WHOLE && NG == 2) {
                const uint32_t v = *reinterpret_cast<const uint32_t *>(sp);
                sc[r][0] = bf16_lo(v);
                sc[r][1 % NG] = bf16_hi(v);
            } else {
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    sc[r][g] = __uint_as_float((uint32_t)sp[min(g, groups - 1 - c * NG)] << 16);
            }
        }
        // four tokens at a time: this lane has values 8 low .. of token 4 i + quad
        const int at = WHOLE ? 8 * low : min(8 * low, a.K - 8 - c * kChunk);
        uint4 *dst = xs + place<GROUP>(low >> 2, low & 3) * 17 + quad;
        if (BF16) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.X) +
                                                        (int64_t)min(4 * i + quad, a.M - 1) * a.K + c * kChunk + at);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * i < a.M)                           // the other rows of the operand are not used
                    dst[4 * i] = make_uint4(perm(x[i].z, x[i].x, 0x05040100u), perm(x[i].z, x[i].x, 0x07060302u),
                                            perm(x[i].w, x[i].y, 0x05040100u), perm(x[i].w, x[i].y, 0x07060302u));
        } else {
            float x[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load8<false>(a.X, (int64_t)min(4 * i + quad, a.M - 1) * a.K + c * kChunk + at, x[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * i >= a.M) break;                   // uniform
                float top = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e += 2) top = fmaxf(top, fmaxf(fabsf(x[i][e]), fabsf(x[i][e + 1])));
                top = group_max(top, 16);
                // top in [2^(e-127), 2^(e-126)): to [2^13, 2^14), or by 2^127
                // where it is below 2^-114
                const int ex = max((int)(__float_as_uint(top) >> 23), 13);
                const float f1 = __uint_as_float((uint32_t)(267 - ex) << 23);
                uint32_t h[4], z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {              // in the codes' order
                    const float v0 = x[i][e] * f1, v1 = x[i][e + 4] * f1;
                    h[e] = f16_pair(v0, v1);
                    z[e] = f16_rest(v0, v1, h[e]);
                }
                dst[4 * i] = make_uint4(h[0], h[1], h[2], h[3]);
                dst[4 * i + 16 * 17] = make_uint4(z[0], z[1], z[2], z[3]);
                if (low == 0) xf[4 * i + quad] = __uint_as_float((uint32_t)(ex - 12) << 23) * 0.5f;   // 2^(ex - 140)
            }
        }
        wave_fence();
        uint4 xr[NS][4];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) xr[s][j] = xs[(s * 16 + j * 4 + quad) * 17 + low];
        const float4v f = *reinterpret_cast<const float4v *>(xf + 4 * quad);
        wave_fence();
        if (!WHOLE && u >= units) {
#pragma unroll
            for (int r = 0; r < R; ++r) w[r] = make_uint4(0, 0, 0, 0);
        }
        float4v x_sum[NG];                      // -24 times the sum of each group's first X, in every column
        const bf8v minus24 = __builtin_bit_cast(bf8v, make_uint4(0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u));
        if (BF16) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                x_sum[g] = float4v{0.f, 0.f, 0.f, 0.f};
                x_sum[g] = mfma_bf16(__builtin_bit_cast(bf8v, xr[0][g * (4 / NG)]), minus24, x_sum[g]);
            }
        }
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
                float4v acc = BF16 ? x_sum[g] : float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = g * (4 / NG); j < (g + 1) * (4 / NG); ++j) {
                    if (BF16) {
                        if (j > g * (4 / NG)) acc = mfma_bf16(__builtin_bit_cast(bf8v, xr[0][j]), minus24, acc);
                        acc = mfma_bf16(__builtin_bit_cast(bf8v, xr[0][j]), codes_to_bf16(d[j]), acc);
                    } else {
                        const half8 b = __builtin_bit_cast(half8, codes_to_f16(d[j]));
#pragma unroll
                        for (int s = 0; s < NS; ++s) acc = mfma_16x16x32(__builtin_bit_cast(half8, xr[s][j]), b, acc);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    tot[r][e] = __builtin_fmaf(BF16 ? acc[e] : acc[e] * f[e], sc[r][g], tot[r][e]);
            }
        }
    }
    __syncthreads();
    float *red = reinterpret_cast<float *>(lds);            // [wave][R][4][64]
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[((wave * R + r) * 4 + e) * 64 + lane] = tot[r][e];
    __syncthreads();
    for (int i = threadIdx.x; i < R * 256; i += blockDim.x) {
        const int r = i >> 8, e = i >> 6 & 3, l = i & 63;
        const int m = 4 * (l >> 4) + e;
        const int64_t n = n0 + 16 * r + (l & 15);
        if (m >= a.M || n >= a.N) continue;
        float y = red[i];
        for (int v = 1; v < waves; ++v) y += red[v * R * 256 + i];
        a.Y[m * (int64_t)a.N + n] = y;
    }
}

// Waves for `parts` of K: as few as keep the longest share of a wave.
int waves_for(int parts, int most) {
    if (parts <= most) return parts > 0 ? parts : 1;
    const int share = (parts + most - 1) / most;
    return (parts + share - 1) / share;
}

template <bool BF16, int M, int R>
void few(const ProdArgs &a, int group, hipStream_t s) {
    const unsigned grid = ((unsigned)a.N + 4 * R - 1) / (4 * R);
    const int waves = waves_for((a.K + kSlice - 1) / kSlice, kMaxWaves);
    hipLaunchKernelGGL((gemv_w4_few_kernel<BF16, M, R>), dim3(grid), dim3(64 * waves), 0, s, a,
                       group == 32 ? 0 : group == 64 ? 1 : 2);
}
template <bool BF16, int M, int R>
void stream(const ProdArgs &a, int group, hipStream_t s) {
    const int tiles = (int)(((unsigned)a.N + 4 * R - 1) / (4 * R)), per = kStreamThreads / 64;
    const int groups = (tiles + per - 1) / per;
    hipLaunchKernelGGL((gemv_w4_stream_kernel<BF16, M, R>),
                       dim3(groups < kStreamGroups ? groups : kStreamGroups), dim3(kStreamThreads),
                       stream_lds(M, a.K), s, a, group == 32 ? 0 : group == 64 ? 1 : 2);
}
template <bool BF16, int GROUP, int R, bool WHOLE, int WAVES>
void many(const ProdArgs &a, hipStream_t s) {
    static_assert(R * 1024 <= wave_lds<BF16>(), "the final sums fit X's place");
    const unsigned grid = ((unsigned)a.N + 16 * R - 1) / (16 * R);
    const int waves = waves_for((a.K + kChunk - 1) / kChunk, WAVES);
    hipLaunchKernelGGL((gemv_w4_mfma_kernel<BF16, GROUP, R, WHOLE, WAVES>), dim3(grid), dim3(64 * waves),
                       waves * wave_lds<BF16>(), s, a);
}
template <bool BF16, int GROUP, bool WHOLE>
void many(const ProdArgs &a, hipStream_t s) {
    // 16 rows a workgroup while each has a CU of its own, then 32, then 64 (the 16
    // waves of a workgroup fill a CU's LDS with fp32 tokens, so one more than 256
    // workgroups is a second turn): 16 x 2560 -> 6912 fp32 (432, 216 and 108 of
    // them) takes 13.4, 8.8 and 12.9 us with R = 1, 2 and 4.  Just above a bound half
    // the CUs have nothing to do.  bf16 tokens, which cost little to bring into the
    // operand's order, go with small workgroups as long as wide ones would be fewer
    // than 1.5 to a CU: 16 x 2560 -> 20000 12.3 us, with R = 4 14.5 (fp32 24.9 and
    // 20.0), 30000 17.5 and 14.7
    if (a.N <= 16 * kCUs) many<BF16, GROUP, 1, WHOLE, 16>(a, s);
    else if (a.N <= 32 * kCUs) many<BF16, GROUP, 2, WHOLE, 16>(a, s);
    else if (BF16 && a.N <= 96 * kCUs) many<BF16, GROUP, 1, WHOLE, 8>(a, s);
    else many<BF16, GROUP, 4, WHOLE, 8>(a, s);
}
template <bool BF16, int GROUP>
void many(const ProdArgs &a, hipStream_t s) {
    if (a.K % kChunk == 0 && reinterpret_cast<uintptr_t>(a.s4) % (2 * kChunk / GROUP) == 0)
        many<BF16, GROUP, true>(a, s);
    else
        many<BF16, GROUP, false>(a, s);
}

template <bool BF16, int M>
void one_or_two(const ProdArgs &a, int group, hipStream_t s) {
    const int from = BF16 ? kStreamRows : kStreamRows / (2 * M);
    // K = 0 has no last unit for the streaming form's loads to clamp to
    if (a.N < from || a.K == 0 || stream_lds(M, a.K) > kStreamLds)
        few<BF16, M, 4>(a, group, s);
    else if (a.N < kWideRows)
        stream<BF16, M, 2>(a, group, s);
    else
        stream<BF16, M, 4>(a, group, s);
}

template <bool BF16>
void product(const ProdArgs &a, int group, hipStream_t s) {
    if (a.M == 1) one_or_two<BF16, 1>(a, group, s);
    else if (a.M == 2) one_or_two<BF16, 2>(a, group, s);
    else if (group == 32) many<BF16, 32>(a, s);
    else if (group == 64) many<BF16, 64>(a, s);
    else many<BF16, 128>(a, s);
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
