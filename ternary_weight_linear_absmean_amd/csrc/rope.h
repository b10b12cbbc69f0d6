// rope.h -- the position rotation of query and key rows.
//
// Pair i of the first `rot` values of a head, (x, y) at (i, i + rot / 2) or at
// (2i, 2i + 1), turns by the angle of row p of cos_sin, [rot / 2 cosines][rot / 2
// sines] in fp32, p the token's position:
//   x' = fl32(x c - y s),  y' = fl32(y c + x s).
// The products of fp32 factors are exact in fp64 and one fused multiply-add
// rounds their sum once to 53 bits, so the result does not depend on how a
// compiler contracts it, and codes formed of it are defined to the bit.  The
// fp64 operations (6 a pair) stay below the time of the rows' bytes.
//
// 4355 fp32 rows of 20 + 5 heads of 128 with the 8-bit append, 118 MB: 23.7 us, 5.0
// TB/s (32.6 with a head to 16 threads, each finding its row's place and loading its
// line of cos_sin; 28.4 with a row to a wave; the rest by stores past the caches).
#pragma once

#include "kv_common.h"

namespace bl {

struct Rope {
    const float *cos_sin;
    int rot;                      // a multiple of 16, <= D; 0: no rotation
    int neighbours;
};

inline Rope rope_device(const bl_rope &r) {
    return {r.cos_sin, (int)r.rot, r.interleaved};
}

// What an append with a rotation takes, on a cache C.
template <class C>
struct Turned {
    Kv8Seqs seqs;
    C c;
    Rope rope;
    const void *k, *v, *q;
    void *q_out;
    int QH;                       // 0: no queries
};
// The same in kFewArgs bytes: what the limits leave free in the counts, and the low
// four bits of the pointers to what is 16-byte aligned, hold the smaller numbers.
struct TurnedArgs {
    const int32_t *q_start, *lengths, *table;
    void *s1, *s2;
    uintptr_t K, V, cos_sin;      // with 12 bits of KVH
    uintptr_t k, v, q, q_out;     // with QH
    int32_t n_tok, n_blocks;
    uint32_t max_blocks : 27, t_shift : 3, neighbours : 1;       // max_blocks T < 2^31, T >= 16
    uint32_t B : 24, rot16 : 4, kvh_top : 4;
};
static_assert(sizeof(TurnedArgs) <= kFewArgs, "a launch's arguments");

template <class C>
inline TurnedArgs packed(const Turned<C> &t) {
    auto with = [](const void *p, int bits) { return reinterpret_cast<uintptr_t>(p) | (uintptr_t)(bits & 15); };
    TurnedArgs a = {t.seqs.q_start, t.seqs.lengths, t.seqs.table, scales1(t.c), scales2(t.c)};
    const int KVH = t.c.KVH, QH = t.QH;
    a.K = with(t.c.K, KVH);
    a.V = with(t.c.V, KVH >> 4);
    a.cos_sin = with(t.rope.cos_sin, KVH >> 8);
    a.kvh_top = (uint32_t)KVH >> 12;
    a.k = with(t.k, QH);
    a.v = with(t.v, QH >> 4);
    a.q = with(QH > 0 ? t.q : nullptr, QH >> 8);
    a.q_out = with(QH > 0 ? t.q_out : nullptr, QH >> 12);
    a.n_tok = t.seqs.n_tok;
    a.n_blocks = t.c.n_blocks;
    a.max_blocks = (uint32_t)t.seqs.max_blocks;
    a.t_shift = (uint32_t)t.c.t_shift;
    a.neighbours = t.rope.neighbours != 0;
    a.B = (uint32_t)t.seqs.B;
    a.rot16 = (uint32_t)t.rope.rot / 16;
    return a;
}
// On the device; an argument that is not packed is as it should be.
template <class C, int D>
__device__ __forceinline__ Turned<C> unpacked(const TurnedArgs &a) {
    // told that it is global memory, as the compiler infers of an argument that is a pointer
    typedef __attribute__((address_space(1))) void global;
    auto address = [](uintptr_t p) { return (void *)(global *)(p & ~(uintptr_t)15); };
    auto bits = [](uintptr_t p) { return (int)(p & 15); };
    Turned<C> t;
    t.seqs = {a.q_start, a.lengths, a.table, a.n_tok, (int)a.B, (int)a.max_blocks};
    const int KVH = bits(a.K) | bits(a.V) << 4 | bits(a.cos_sin) << 8 | (int)a.kvh_top << 12;
    t.c = cache_of<C>(address(a.K), address(a.V), a.s1, a.s2, a.n_blocks, KVH, (int)a.t_shift, D);
    t.rope = {static_cast<const float *>(address(a.cos_sin)), (int)a.rot16 * 16, (int)a.neighbours};
    t.k = address(a.k);
    t.v = address(a.v);
    t.q = address(a.q);
    t.q_out = address(a.q_out);
    t.QH = bits(a.k) | bits(a.v) << 4 | bits(a.q) << 8 | bits(a.q_out) << 12;
    return t;
}
template <class C, int D, class A>
__device__ __forceinline__ const A &unpacked(const A &a) { return a; }

// Rows that this kernel does not read again: past the caches.
__device__ __forceinline__ void store_row4(float *p, float4 v) {
    __builtin_nontemporal_store(float4v{v.x, v.y, v.z, v.w}, reinterpret_cast<float4v *>(p));
}
__device__ __forceinline__ void store_row4(uint16_t *p, float4 v) {
    typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(uint2v{bf16_round(v.x) | bf16_round(v.y) << 16, bf16_round(v.z) | bf16_round(v.w) << 16},
                                reinterpret_cast<uint2v *>(p));
}

// x c - y s (or + with s negated), rounded once to fp32.
__device__ __forceinline__ float turned(float x, float c, float y, float s) {
    return (float)__builtin_fma((double)x, (double)c, -((double)y * (double)s));
}

__device__ __forceinline__ float4 load_row4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load_row4(const uint16_t *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

// N pieces of four values: piece i is values d[i] .. d[i] + 3 of the head at
// rows[i], turned for position pos[i], as it is where that is below 0 or d[i] not
// below rot.  Every load is issued before the first is used, at clamped places.
template <int N, typename E>
__device__ __forceinline__ void load_turned(const E *const *rows, const int *d, const int64_t *pos,
                                            const Rope &rope, float4 *v) {
    const int half = rope.rot / 2;
    float4 y[N], c[N], s[N];
    if (rope.neighbours) {                                        // uniform
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool on = pos[i] >= 0 && d[i] < rope.rot;
            const float *line = rope.cos_sin + (on ? pos[i] : 0) * rope.rot + (on ? d[i] : 0) / 2;
            v[i] = load_row4(rows[i] + d[i]);
            const float2 c2 = *reinterpret_cast<const float2 *>(line);
            const float2 s2 = *reinterpret_cast<const float2 *>(line + half);
            c[i] = make_float4(c2.x, c2.x, c2.y, c2.y);
            s[i] = make_float4(s2.x, -s2.x, s2.y, -s2.y);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = make_float4(v[i].y, v[i].x, v[i].w, v[i].z);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool on = pos[i] >= 0 && d[i] < rope.rot;
            const int at = on ? d[i] : 0;
            const float *line = rope.cos_sin + (on ? pos[i] : 0) * rope.rot + (at < half ? at : at - half);
            v[i] = load_row4(rows[i] + d[i]);
            y[i] = load_row4(rows[i] + (at < half ? at + half : at - half));
            c[i] = load_row4(line);
            s[i] = load_row4(line + half);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (d[i] >= half) s[i] = make_float4(-s[i].x, -s[i].y, -s[i].z, -s[i].w);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool on = pos[i] >= 0 && d[i] < rope.rot;
        const float4 x = v[i];
        const float4 r = make_float4(turned(x.x, c[i].x, y[i].x, s[i].x), turned(x.y, c[i].y, y[i].y, s[i].y),
                                     turned(x.z, c[i].z, y[i].z, s[i].z), turned(x.w, c[i].w, y[i].w, s[i].w));
        v[i] = on ? r : x;
    }
}

// The same for 8 values of several heads at one position: d .. d + 7, in range.
struct Turn8 {
    float4 c[2], s[2];
    int other = -1;               // where the second half of the pairs stands; -1: among the values
    __device__ __forceinline__ Turn8() {}
    __device__ __forceinline__ Turn8(const Rope &rope, int64_t pos, int d) {
        const int half = rope.rot / 2;
        const float *line = rope.cos_sin + pos * rope.rot;
        if (rope.neighbours) {                                    // uniform
            other = -1;
            const float4 c4 = load_row4(line + d / 2), s4 = load_row4(line + half + d / 2);
            c[0] = make_float4(c4.x, c4.x, c4.y, c4.y);
            c[1] = make_float4(c4.z, c4.z, c4.w, c4.w);
            s[0] = make_float4(s4.x, -s4.x, s4.y, -s4.y);
            s[1] = make_float4(s4.z, -s4.z, s4.w, -s4.w);
        } else {
            const bool upper = d >= half;
            const int at = upper ? d - half : d;
            other = upper ? at : d + half;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                c[i] = load_row4(line + at + 4 * i);
                s[i] = load_row4(line + half + at + 4 * i);
                if (upper) s[i] = make_float4(-s[i].x, -s[i].y, -s[i].z, -s[i].w);
            }
        }
    }
    template <typename E>
    __device__ __forceinline__ void load_others(const E *row, float4 *y) const {
        if (other < 0) return;                                    // uniform
        y[0] = load_row4(row + other);
        y[1] = load_row4(row + other + 4);
    }
    __device__ __forceinline__ void apply(float4 *x, float4 *y) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = x[i], w = other < 0 ? make_float4(v.y, v.x, v.w, v.z) : y[i];
            x[i] = make_float4(turned(v.x, c[i].x, w.x, s[i].x), turned(v.y, c[i].y, w.y, s[i].y),
                               turned(v.z, c[i].z, w.z, s[i].z), turned(v.w, c[i].w, w.w, s[i].w));
        }
    }
};

// The query rows of a call, turned: a wave to a row, 8 values a lane, D / 8 lanes
// to a head, the row's heads in turn, so that a row's place and its line of cos_sin are
// found and loaded once.  Rows of no sequence are left; a row whose position
// the cache has no room for is copied as it is.
// A wave takes all heads of a row, or in calls of few rows those of one step: a
// decode step waits for one wave's chain of loads, a prompt for the bytes.
constexpr int64_t kFewTurnedRows = 512;
constexpr int rope_heads(int64_t n_tok, int64_t QH, int64_t D) {
    return n_tok > kFewTurnedRows ? (int)QH : (int)(512 / D);
}
constexpr int64_t rope_groups(int64_t n_tok, int64_t QH, int64_t D, int threads) {
    if (QH == 0) return 0;
    const int64_t per = rope_heads(n_tok, QH, D), waves = n_tok * ((QH + per - 1) / per);
    return (waves + threads / 64 - 1) / (threads / 64);
}
template <int AT_ONCE, typename E>
__device__ __forceinline__ void turn_heads(const E *q, E *out, int64_t row0, int h0, int h1, int step, int d_shift,
                                           int d, bool on, const Turn8 &turn) {
    for (; h0 < h1; h0 += AT_ONCE * step) {
        float4 x[AT_ONCE][2], y[AT_ONCE][2];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {                       // all loads in flight, at clamped places
            const E *src = q + ((row0 + min(h0 + i * step, h1 - 1)) << d_shift);
            x[i][0] = load_row4(src + d);
            x[i][1] = load_row4(src + d + 4);
            turn.load_others(src, y[i]);
        }
        // out may be q: a head's threads are lanes of one wave, all of whose loads
        // stand before its first store, and its heads are read by no other wave
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int h = h0 + i * step;
            if (h >= h1) continue;
            if (on) turn.apply(x[i], y[i]);
            E *dst = out + ((row0 + h) << d_shift) + d;
            store_row4(dst, x[i][0]);
            store_row4(dst + 4, x[i][1]);
        }
    }
}
template <int THREADS, typename E>
__device__ __forceinline__ void turn_queries(const E *q, E *out, int QH, int per, int d_shift, const Kv8Seqs &seqs,
                                             int64_t room, const Rope &rope, int64_t group) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = group * (THREADS >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = (QH + per - 1) / per;
    const int64_t row = unit / chunks;
    const int first = (int)(unit - row * chunks) * per, h1 = min(first + per, QH);
    if (row >= seqs.n_tok) return;                                // uniform
    const SeqPlace in = find_place(seqs, row, [](int q, int) { return (int64_t)q; });
    if (row < in.q0 || row >= in.q1) return;
    int64_t pos = (int64_t)in.length - (in.q1 - row);
    if (pos >= room) pos = -1;
    const int per_shift = d_shift - 3, step = 64 >> per_shift;    // lanes of a head, heads at once
    const int d = 8 * (lane & ((1 << per_shift) - 1));
    const bool on = pos >= 0 && d < rope.rot;
    Turn8 turn;
    if (room > 0) turn = Turn8(rope, on ? pos : 0, on ? d : 0);   // uniform; a cache without room has no cos_sin
    if (h1 - first <= step)
        turn_heads<1>(q, out, row * QH, first + (lane >> per_shift), h1, step, d_shift, d, on, turn);
    else
        turn_heads<4>(q, out, row * QH, first + (lane >> per_shift), h1, step, d_shift, d, on, turn);
}

}  // namespace bl
