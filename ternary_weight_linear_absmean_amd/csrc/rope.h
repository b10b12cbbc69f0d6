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

// The query rows of a call, turned: workgroup `group` of THREADS takes 8 values
// a thread of the line of all.  Rows of no sequence are left; a row whose
// position the cache has no room for is copied as it is.
template <int THREADS>
constexpr int64_t rope_groups(int64_t n_tok, int64_t QH, int64_t D) {
    return (n_tok * QH * D / 8 + THREADS - 1) / THREADS;
}
__device__ __forceinline__ void store_row4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store_row4(uint16_t *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(bf16_round(v.x) | bf16_round(v.y) << 16, bf16_round(v.z) | bf16_round(v.w) << 16);
}
template <int THREADS, typename E>
__device__ __forceinline__ void turn_queries(const E *q, E *out, int QH, int d_shift, const Kv8Seqs &seqs,
                                             int64_t room, const Rope &rope, int64_t group) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int per_shift = d_shift - 3;                            // threads of a head
    const int64_t heads = (int64_t)seqs.n_tok * QH;
    const int64_t first = (group * THREADS + wave * 64) >> per_shift;      // a wave's heads
    if (first >= heads) return;                                   // uniform
    const int64_t head = first + (lane >> per_shift);
    const int64_t last = min(first + (64 >> per_shift), heads) - 1;
    const int row0 = (int)(first / QH), row1 = (int)(last / QH);
    const int row = head < heads ? (int)(head / QH) : row1;
    int64_t pos = -1;
    bool mine = false;
    for (int r = row0; r <= row1; ++r) {                          // one row of most calls, eight at most
        const int b = find_seq(seqs.B, r, [&](int i) { return (int64_t)q_at(seqs, i); });
        const int q0 = q_at(seqs, b), q1 = q_at(seqs, b + 1);
        if (r == row && r >= q0 && r < q1) {
            mine = true;
            pos = (int64_t)seqs.lengths[b] - (q1 - r);
        }
    }
    if (!mine || head >= heads) return;
    const int d = 8 * (lane & ((1 << per_shift) - 1));
    const E *const src = q + (head << d_shift), *rows[2] = {src, src};
    if (pos >= room) pos = -1;
    const int at[2] = {d, d + 4};
    const int64_t place[2] = {pos, pos};
    float4 v[2];
    load_turned<2>(rows, at, place, rope, v);
    // out may be q: a head's threads are lanes of one wave, all of whose loads
    // stand before its first store
    __builtin_amdgcn_wave_barrier();
    store_row4(out + (head << d_shift) + d, v[0]);
    store_row4(out + (head << d_shift) + d + 4, v[1]);
}

}  // namespace bl
