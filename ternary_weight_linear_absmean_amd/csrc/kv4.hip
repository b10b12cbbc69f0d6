// kv4.hip -- new key / value rows into the 4-bit cache, keys and queries turned
// by their positions on the way.
//
// Per token and head, for K and for V apart, over the D values x (within
// +-65504, the largest fp16; what is beyond counts as that, NaN as -65504):
//   z = the largest fp16 <= min x,  s = fp16(fl(fl(max x - z) / 15)),
//   code = clamp(rne(fl(fl(x - z) / s)), 0, 15), 0 where s = 0;
// the value is z + s code.  z is rounded down so that no value lies below the
// first code.  A step that is rounded down costs the largest value 15 times that: at
// most 15 / 2048 of a step, or, where the spread is below 15 2^-14 = 9.2e-4 and fp16 holds
// s in steps of 2^-24, at most 15 2^-25 = 4.5e-7, which can be several of its steps.  So
// a value is off by max(s / 2, 4.5e-7).  Scales of a token, not of a block: 4-bit codes do not survive
// being rescaled when a block's largest value grows.  Quotients are correctly
// rounded, so the cache's bytes are defined to the bit.
//
// One workgroup per (16 consecutive positions of a sequence, head): 16
// tokens' codes of one value of V are the 8 bytes of a group, so it alone writes
// them, also where it brings a single token and the others' codes stay.  D / 8
// threads to a token, 8 values each.  The grid is known without the lengths:
// sequence b with n_b new tokens touches at most ceil(n_b / 16) + 1 such groups,
// and the slots first(b) = floor(q_start[b] / 16) + 2 b leave it no fewer.
//
// Decode is bound by latency: starts and length, table entry beside the rows and
// the line of cos_sin, minimum and maximum, quotients, one after the other (64
// sequences, 5 heads of 4, D = 128, bf16, queries turned too: 5.9 us on the GPU, 5.3 as they
// are).  Prompts are one pass over the rows, the queries' part the larger (4355 rows, 8
// heads of 2, D = 64, fp32: 54 MB in 14.2 us, 3.8 TB/s).  4209 rows of 5 heads of 4, D =
// 128, three sequences: bf16 59 MB in 20.5 us, fp32 113 MB in 26.4; without rotation 13.6 MB
// in 9.1 and 24.4 MB in 10.0, a workgroup's chain.
#include "kv4_common.h"
#include "rope.h"

#include <type_traits>

namespace bl {
namespace {

constexpr int kTokens = 16;       // of a workgroup

// The largest fp16 that is at most x, |x| <= 65504.
__device__ __forceinline__ _Float16 f16_below(float x) {
    const _Float16 h = (_Float16)x;
    const uint16_t w = __builtin_bit_cast(uint16_t, h);
    const uint16_t down = (w & 0x7FFF) == 0 ? 0x8001 : w & 0x8000 ? w + 1 : w - 1;
    return (float)h > x ? __builtin_bit_cast(_Float16, down) : h;
}

struct Args {
    Kv8Seqs seqs;
    Kv4Cache c;
    const void *k, *v;
};

// Eight values of a row, and with those of the row's other threads its z and s and
// these values' codes.
template <int PER>
__device__ __forceinline__ uint32_t quantised(const float4 *x, uint32_t *u) {
    float f[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    float lo = 65504.0f, hi = -65504.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f[e] = fminf(fmaxf(f[e], -65504.0f), 65504.0f);
        lo = fminf(lo, f[e]);
        hi = fmaxf(hi, f[e]);
    }
    lo = -group_max(-lo, PER);
    hi = group_max(hi, PER);
    const _Float16 z = f16_below(lo);
    const float zf = (float)z;
    const _Float16 step = (_Float16)__fdiv_rn(__fsub_rn(hi, zf), 15.0f);
    const float sf = (float)step;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float r = __builtin_rintf(__fdiv_rn(__fsub_rn(f[e], zf), sf));
        u[e] = sf > 0.0f ? (uint32_t)fminf(fmaxf(r, 0.0f), 15.0f) : 0u;
    }
    return __builtin_bit_cast(uint32_t, half2{z, step});
}

template <typename E, int D, bool ROPE>
__global__ __launch_bounds__(2 * D) void kv4_append_kernel(std::conditional_t<ROPE, TurnedArgs, Args> given) {
    constexpr int kPer = D / 8;                           // threads of a token
    __shared__ alignas(16) uint8_t codes[D][kTokens];
    const auto &a = unpacked<Kv4Cache, D>(given);
    const Kv8Seqs &seqs = a.seqs;
    const Kv4Cache &c = a.c;
    if constexpr (ROPE) {
        const int64_t appends = ((seqs.n_tok >> 4) + 2 * (int64_t)seqs.B) * c.KVH;
        if (blockIdx.x >= appends) {
            turn_queries<2 * D>(static_cast<const E *>(a.q), static_cast<E *>(a.q_out), a.QH,
                                rope_heads(seqs.n_tok, a.QH, D), D == 64 ? 6 : 7, seqs,
                                (int64_t)seqs.max_blocks << c.t_shift, a.rope, blockIdx.x - appends);
            return;
        }
    }
    const uint32_t slot = blockIdx.x / (uint32_t)c.KVH;
    const int h = (int)(blockIdx.x - slot * c.KVH);
    const SeqPlace in_seq = find_place(seqs, slot, [](int q, int i) { return (int64_t)(q >> 4) + 2 * (int64_t)i; });
    const int b = in_seq.b, q0 = in_seq.q0, n = in_seq.q1 - q0;
    const int64_t nth = (int64_t)slot - ((q0 >> 4) + 2 * (int64_t)b);
    if (nth < 0 || n <= 0) return;
    const int64_t len = in_seq.length, start = len - n;            // of row q0
    const int64_t j = (max(start, (int64_t)0) >> 4) + nth;         // the sequence's group
    const int64_t first = max(max(start, (int64_t)0), 16 * j), last = min(len, 16 * j + 16);
    if (j >= (int64_t)seqs.max_blocks << c.t_shift >> 4 || first >= last) return;
    const int id = seqs.table[(int64_t)b * seqs.max_blocks + (16 * j >> c.t_shift)];

    // this thread's token and values; slots without a new token repeat the first
    const int t = threadIdx.x / kPer, td = threadIdx.x % kPer;
    const bool mine = 16 * j + t >= first && 16 * j + t < last;
    const int64_t pos = mine ? 16 * j + t : first;
    const int64_t row = ((q0 + (pos - start)) * c.KVH + h) * (int64_t)D;
    const E *const k = static_cast<const E *>(a.k) + row, *const v = static_cast<const E *>(a.v) + row;
    float4 x[2], y[2], w[2];
    x[0] = load_row4(k + 8 * td);
    x[1] = load_row4(k + 8 * td + 4);
    w[0] = load_row4(v + 8 * td);
    w[1] = load_row4(v + 8 * td + 4);
    if constexpr (ROPE) {
        const bool on = 8 * td < a.rope.rot;
        const Turn8 turn(a.rope, pos, on ? 8 * td : 0);
        turn.load_others(k, y);
        if (on) turn.apply(x, y);
    }
    if (id < 0 || id >= c.n_blocks) return;                        // uniform: the block holds no token
    const int64_t head = (int64_t)id * c.KVH + h, token = head * c.T + (pos & (c.T - 1));
    uint8_t *const group = c.V + (head * (c.T / 16) + (j & (c.T / 16 - 1))) * (int64_t)(8 * D);
    const int s0 = (int)(first - 16 * j), s1 = (int)(last - 16 * j);
    const bool whole = s1 - s0 == kTokens;
    uint2 old = make_uint2(0u, 0u);
    if (!whole && threadIdx.x < D) old = *reinterpret_cast<const uint2 *>(group + 8 * threadIdx.x);

    uint32_t u[8];
    const uint32_t zk = quantised<kPer>(x, u);
    if (mine) {
        uint32_t p = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) p |= u[e] << (4 * e);
        *reinterpret_cast<uint32_t *>(c.K + token * (D / 2) + 4 * td) = p;
    }
    const uint32_t zv = quantised<kPer>(w, u);
    if (mine && td == 0) {
        c.zk[token] = zk;
        c.zv[token] = zv;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) codes[8 * td + e][t] = (uint8_t)u[e];
    __syncthreads();
    if (threadIdx.x >= D) return;
    const uint4 g = *reinterpret_cast<const uint4 *>(codes[threadIdx.x]);
    // bytes 0 n 0 n -> nibbles
    auto pack = [](uint32_t lo4, uint32_t hi4) {
        const uint32_t p = lo4 | lo4 >> 4, r = hi4 | hi4 >> 4;
        return perm(r, p, 0x06040200u);
    };
    uint2 fresh = make_uint2(pack(g.x, g.y), pack(g.z, g.w));
    if (!whole) {
        const uint64_t keep = ~((~0ull >> (64 - 4 * (s1 - s0))) << (4 * s0));
        fresh.x = (old.x & (uint32_t)keep) | (fresh.x & ~(uint32_t)keep);
        fresh.y = (old.y & (uint32_t)(keep >> 32)) | (fresh.y & ~(uint32_t)(keep >> 32));
    }
    *reinterpret_cast<uint2 *>(group + 8 * threadIdx.x) = fresh;
}

template <typename E, int D>
hipError_t append(const void *k, const void *v, const void *q, void *q_out, int QH, const Kv8Seqs &seqs,
                  const Kv4Cache &c, const Rope *rope, hipStream_t s) {
    // of 16 positions; then the queries' workgroups
    int64_t groups = ((seqs.n_tok >> 4) + 2 * (int64_t)seqs.B) * c.KVH;
    if (rope) groups += rope_groups(seqs.n_tok, QH, D, 2 * D);
    if (groups * 2 * D >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
    if (rope) {
        const TurnedArgs a = packed(Turned<Kv4Cache>{seqs, c, *rope, k, v, q, q_out, QH});
        hipLaunchKernelGGL((kv4_append_kernel<E, D, true>), dim3((unsigned)groups), dim3(2 * D), 0, s, a);
    } else {
        const Args a = {seqs, c, k, v};
        static_assert(sizeof a <= kFewArgs, "a launch's arguments");
        hipLaunchKernelGGL((kv4_append_kernel<E, D, false>), dim3((unsigned)groups), dim3(2 * D), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_append(const void *k, const void *v, const void *q, void *q_out, int dtype, int QH,
                             const Kv8Seqs &seqs, const bl_kv4 &cache, const bl_rope *rope, hipStream_t s) {
    const Kv4Cache c = kv4_device(cache);
    Rope r = {};
    if (rope) r = rope_device(*rope);
    const Rope *rp = rope ? &r : nullptr;
    if (c.D == 64)
        return dtype ? append<uint16_t, 64>(k, v, q, q_out, QH, seqs, c, rp, s)
                     : append<float, 64>(k, v, q, q_out, QH, seqs, c, rp, s);
    return dtype ? append<uint16_t, 128>(k, v, q, q_out, QH, seqs, c, rp, s)
                 : append<float, 128>(k, v, q, q_out, QH, seqs, c, rp, s);
}

}  // namespace bl
