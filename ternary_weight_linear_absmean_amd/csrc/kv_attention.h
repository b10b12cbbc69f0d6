// kv_attention.h -- what the attentions over the paged caches share: who reads
// which keys, the join of a row's parts, and what a call launches.  C is the
// cache's device view, Kv8Cache or Kv4Cache.
#pragma once

#include "kv_common.h"

namespace bl {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kCUs = 256;
constexpr int kTile = 64;                   // keys per wave and step
constexpr int kRows = 16;                   // rows of a tile
constexpr int kFewRows = 32;                // rows of a sequence above which they are many
constexpr int kFewTiles = kFewRows / kRows;
constexpr int kGroups = 512;               // workgroups of 256 that run at once: two to a CU
constexpr int kStepShift = 8;               // log2 of the keys that a workgroup's waves take in a step
constexpr int kMaxParts = kGroups;
constexpr int kManyWork = 4500;             // see Plan
constexpr int kLongSteps = 32;              // see Plan
constexpr int kLineSeqs = 256;              // sequences that a wave lines up, four to a lane

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Four consecutive values of a row.
template <bool BF16>
__device__ __forceinline__ float4 load4(const void *p, int64_t at) {
    if (BF16) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at);
        return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    }
    return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
}
template <bool BF16>
__device__ __forceinline__ void store4(void *p, int64_t at, float4 v) {
    if (BF16) {
        uint2 w;
        w.x = bf16_round(v.x) | bf16_round(v.y) << 16;
        w.y = bf16_round(v.z) | bf16_round(v.w) << 16;
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + at) = w;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + at) = v;
    }
}

// A power of two >= |x| (for |x| in [2^-100, 2^126)); 2^14 over it stays finite.
__device__ __forceinline__ float pow2_above(float x) {
    const uint32_t e = min(max((__float_as_uint(x) >> 23) & 255u, 27u), 252u);
    return __uint_as_float((e + 1) << 23);
}

// 1 / x for a power of two in [2^-126, 2^126].
__device__ __forceinline__ float pow2_inverse(float x) {
    return __uint_as_float(0x7F000000u - __float_as_uint(x));
}

// The power of two that takes |x| <= top to [2^13, 2^14), or 2^127 where top is
// below 2^-114.
__device__ __forceinline__ float to_f16_range(float top) {
    const int e = max((int)(__float_as_uint(top) >> 23), 13);
    return __uint_as_float((uint32_t)(267 - e) << 23);
}

constexpr float kUnit = 16384.0f;           // p sv / u is held as fp16 times this
// A row's reference m follows its maximum only when that is kSlack above it:
// 2^kSlack kUnit still is in fp16's range, and with scores of one spread the
// sums are rescaled once or twice a sequence and not at every step.
constexpr float kSlack = 1.9f;
// That bound needs the scores' rounding to be small: the maximum is taken of
// rounded products, the exponent of the unrounded (one multiply-add), and m +
// kSlack is rounded too, by half a step of a number next to m each: 2^-5 in all
// at |m| = 2^18, and 2^1.94 kUnit < 62900 < 65504.  bf16 rows' exponent has the
// value scale in it, rounded with m: 2^-14 at 2^11, a quarter of what rounding
// the weight to 11 bits takes.  From there on m follows every maximum, and the
// scores are rounded and m is taken off them before the exponent is formed, so
// that the largest weight is 1 and a value scale costs nothing.  Such scores cost
// 1 to 3% (2 prompts of 2048 and 1500 bf16 rows 166 and 170 us, 64 ragged
// sequences of up to 4096 keys 43.3 and 43.8).
template <bool BF16>
constexpr float kFarScore = BF16 ? 2048.0f : 262144.0f;
template <bool BF16>
__device__ __forceinline__ float raise_above(float m) {     // a maximum that makes m follow
    return fabsf(m) < kFarScore<BF16> ? m + kSlack : -INFINITY;
}
constexpr float kTiny = 1.17549435e-38f;    // a score factor of 0 (or none) without 0 * inf

// A count of keys taken into [0, most].
__device__ __forceinline__ uint32_t keys_within(int64_t keys, uint32_t most) {
    return (uint32_t)min(max(keys, (int64_t)0), (int64_t)most);
}

template <class C>
struct KvArgs {
    const void *q;
    void *out;
    Kv8Seqs seqs;
    C c;
    int QH, G;
    float scale2;             // scale * log2(e)
    // rows of the sequences that a kernel takes: more than, at most
    int64_t min_rows, max_rows;
    bool mixed;               // both kernels run
    // many rows: up to S parts of a sequence's keys; [S][n_tok * QH][D], then
    // [S][n_tok * QH][2]
    float *part;
    int S;
    int64_t many_groups;      // workgroups of a part
    // few rows: pieces for about `most` workgroups; cuts: whether a unit may be
    // cut, `slots` pieces of such at most; [slots][16][D], then [slots][16][2],
    // then (slot and row of the first, pieces) by row of q
    float *cut;
    int most, slots, step_shift;
    bool cuts;
};

template <class C>
__device__ __forceinline__ int64_t key_capacity(const KvArgs<C> &a) {
    return a.c.n_blocks > 0 ? (int64_t)a.seqs.max_blocks << a.c.t_shift : 0;
}

// Who reads which keys, for few rows.  A unit is (16 rows of a sequence, key
// head) over the sequence's keys, in steps of 256 keys (64 of each wave).  The
// lengths are on the device, so every workgroup works the division out from
// them, the same for all: U units of W steps in all are cut into pieces of c =
// ceil(W / most) steps; that makes W / c + U pieces at most, 2 W / c of them of
// units that are cut.  Workgroup i takes piece i of the line of all.
//
// Nothing is cut where that saves the longest unit less than three steps (1.7
// us each when they wait for memory), as the join is a launch and 2 to 3 us, nor
// where U >= most / 2 and the longest has less than 2.5 c: then the units fill
// the GPU evenly enough.  64 ragged sequences of up to 4096 keys, 5 heads: 48.1
// us uncut, 42.3 cut; 96 of them 63 and 67, 128 73 and 80.  Units of about one
// length get as many pieces as keep all within `most`, since a few more would
// run alone at the end (32 sequences of 4096 keys: 3 pieces of 6 steps 39.4 us,
// 4 of 5 44.0; ragged, 25).  With max_blocks in the lengths' place 2000 keys with
// room for 32768 took 12.3 us and not 9.1, 16 x 4000 with room for 131072 37 and
// not 22, 63 x 500 beside 20000 150 and not 20.
//
// With more than kLineSeqs sequences nothing is cut and a unit's place follows
// from q_start alone: tile slots of sequence b from floor(q_start[b] G / 16) + b
// on, or, where sequences of more than kFewRows go to the other kernel, the two
// that kFewRows make; KVH units each.  (Slots leave some workgroups idle, a
// fifth with 4 rows a sequence: 64 ragged sequences of up to 4096 keys 54.4 us,
// in a line 48.1; in a line of 1000 sequences every workgroup would look at all
// of them: 250 keys each 73.8 and 128 us.)
template <class C>
__device__ __forceinline__ int2 *cut_info(const KvArgs<C> &a, int D) {
    return reinterpret_cast<int2 *>(a.cut + (int64_t)a.slots * kRows * (D + 2));
}
template <class C>
__device__ __forceinline__ uint32_t steps_of(const KvArgs<C> &a, int length, int shift) {
    const int64_t keys = min(max((int64_t)length, (int64_t)1), max(key_capacity(a), (int64_t)1));
    return (uint32_t)((keys - 1) >> shift) + 1;
}
struct SeqWork {
    int q0, n, length;
    uint32_t tiles, steps;
};
template <class C>
__device__ __forceinline__ SeqWork work_of(const KvArgs<C> &a, int q0, int q1, int length) {
    SeqWork w;
    w.q0 = min(max(q0, 0), a.seqs.n_tok);
    w.n = min(max(q1, 0), a.seqs.n_tok) - w.q0;
    w.length = length;
    const int64_t rows = (int64_t)w.n * a.G;
    w.tiles = rows > 0 && rows <= a.max_rows ? (uint32_t)(rows + kRows - 1) / kRows : 0u;
    w.steps = steps_of(a, length, a.step_shift);
    return w;
}
template <class C>
__device__ __forceinline__ SeqWork work_of(const KvArgs<C> &a, int b) {
    return work_of(a, a.seqs.q_start[b], a.seqs.q_start[b + 1], a.seqs.lengths[b]);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_0(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
// Running sum / maximum over the lanes: row_shr 1, 2, 4, 8, then the last lane
// of each 16 to the next, of the first 32 to the others.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    v += dpp_or_0<0x111, 0xF>(v);
    v += dpp_or_0<0x112, 0xF>(v);
    v += dpp_or_0<0x114, 0xF>(v);
    v += dpp_or_0<0x118, 0xF>(v);
    v += dpp_or_0<0x142, 0xA>(v);
    v += dpp_or_0<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ uint32_t wave_scan_max(uint32_t v) {
    v = max(v, dpp_or_0<0x111, 0xF>(v));
    v = max(v, dpp_or_0<0x112, 0xF>(v));
    v = max(v, dpp_or_0<0x114, 0xF>(v));
    v = max(v, dpp_or_0<0x118, 0xF>(v));
    v = max(v, dpp_or_0<0x142, 0xA>(v));
    return max(v, dpp_or_0<0x143, 0xC>(v));
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

template <class C>
__device__ __forceinline__ uint32_t steps_of_piece(const KvArgs<C> &a, uint32_t units, uint32_t steps, uint32_t top) {
    const uint32_t most = (uint32_t)a.most;
    uint32_t c = max((steps + most - 1) / most, 1u);
    // W / c <= most either way
    if (units > 0 && top * units - steps <= steps / 4) {
        const uint32_t each = max(most / units, 1u);
        c = max((top + each - 1) / each, 1u);
    }
    return top < c + 3 || (2 * units >= most && 2 * top < 5 * c) ? top : c;
}

// Piece `pos` of the line: which of its unit, and where among the pieces of
// units that are cut the unit's begin (-1: not cut).
struct Piece {
    SeqWork work;
    int b, slot;
    uint32_t h, tile, nth, pieces, c;       // head and 16 rows; of the unit's pieces, of c steps
};
template <class C>
__device__ __forceinline__ bool find_unit(const KvArgs<C> &a, uint32_t pos, Piece &p) {
    const int64_t slot = pos / (uint32_t)a.c.KVH;
    p.h = pos - (uint32_t)slot * a.c.KVH;
    int64_t nth;
    if (a.mixed) {
        p.b = (int)(slot / kFewTiles);
        nth = slot % kFewTiles;
    } else {
        p.b = find_seq(a.seqs.B, slot, [&](int i) { return (int64_t)q_at(a.seqs, i) * a.G / kRows + i; });
        nth = slot - ((int64_t)q_at(a.seqs, p.b) * a.G / kRows + p.b);
    }
    p.work = work_of(a, p.b);
    p.tile = (uint32_t)nth;
    p.nth = 0;
    p.pieces = 1;
    p.slot = -1;
    return nth >= 0 && nth < p.work.tiles;
}
template <class C>
__device__ __forceinline__ bool find_piece(const KvArgs<C> &a, uint32_t pos, Piece &p) {
    const int lane = threadIdx.x & 63, B = a.seqs.B;
    const uint32_t heads = (uint32_t)a.c.KVH;
    uint32_t cut_before = 0;
    if (B == 1) {
        p.b = 0;
        p.work = work_of(a, 0);
        const uint32_t units = heads * p.work.tiles;
        p.pieces = 1;
        if (a.cuts) {
            p.c = steps_of_piece(a, units, units * p.work.steps, p.work.steps);
            p.pieces = (p.work.steps + p.c - 1) / p.c;
        }
        if (pos >= units * p.pieces) return false;
    } else {
        constexpr int kPer = kLineSeqs / 64;     // sequence 64 j + lane
        int q0[kPer], q1[kPer], length[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            q0[j] = q1[j] = length[j] = 0;
            if (64 * j < B) {
                const int b = min(64 * j + lane, B - 1);
                q0[j] = a.seqs.q_start[b];
                q1[j] = a.seqs.q_start[b + 1];
                length[j] = a.seqs.lengths[b];
            }
        }
        SeqWork w[kPer];
        uint32_t units = 0, steps = 0, top = 1;
        p.c = 0xFFFFFFFFu;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            w[j] = work_of(a, q0[j], q1[j], length[j]);
            if (64 * j + lane >= B) w[j].tiles = 0;
            const uint32_t u = heads * w[j].tiles;
            units += u;
            steps += u * w[j].steps;
            top = max(top, u > 0 ? w[j].steps : 1u);
        }
        if (a.cuts)
            p.c = steps_of_piece(a, lane_of(wave_scan(units), 63), lane_of(wave_scan(steps), 63),
                                 lane_of(wave_scan_max(top), 63));
        bool found = false;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (64 * j >= B || found) continue;             // uniform
            const uint32_t pieces = w[j].steps <= p.c ? 1u : (w[j].steps + p.c - 1) / p.c;
            const uint32_t mine = heads * w[j].tiles * pieces, cut = pieces > 1 ? mine : 0u;
            const uint32_t upto = wave_scan(mine), cut_upto = a.cuts ? wave_scan(cut) : 0u;
            const uint64_t in = __ballot(pos < upto);
            if (in != 0) {
                const int i = __builtin_ctzll(in);
                found = true;
                pos -= lane_of(upto - mine, i);
                cut_before += lane_of(cut_upto - cut, i);
                p.b = 64 * j + i;
                p.pieces = lane_of(pieces, i);
                p.work = SeqWork{(int)lane_of((uint32_t)w[j].q0, i), (int)lane_of((uint32_t)w[j].n, i),
                                 (int)lane_of((uint32_t)w[j].length, i), lane_of(w[j].tiles, i),
                                 lane_of(w[j].steps, i)};
            } else {
                pos -= lane_of(upto, 63);
                cut_before += lane_of(cut_upto, 63);
            }
        }
        if (!found) return false;
    }
    const uint32_t unit = p.pieces == 1 ? pos : pos / p.pieces;
    p.nth = pos - unit * p.pieces;
    // tiles that see most first, so that what starts last is short (4-bit cache, fp32:
    // 1024 rows on their own keys, 5 heads of 4, 35.5 us, so 29.8)
    const uint32_t back = p.work.tiles == 1 ? 0u : unit / heads;
    p.tile = p.work.tiles - 1 - back;
    p.h = unit - back * heads;
    p.slot = p.pieces == 1 ? -1 : (int)(cut_before + unit * p.pieces);
    return true;
}

constexpr int kManyRows = 128;
typedef float float16v __attribute__((ext_vector_type(16)));
__device__ __forceinline__ float16v mfma_32x32x16(half8 a, half8 b, float16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
// Keys of a part of a sequence: a S-th of them in whole steps, or all where
// that saves fewer than three.
template <class C>
__device__ __forceinline__ int64_t keys_of_part(const KvArgs<C> &a, int length) {
    const uint32_t steps = steps_of(a, length, kStepShift), each = (steps + a.S - 1) / (uint32_t)a.S;
    return (int64_t)(steps - each < 3 ? steps : each) << kStepShift;
}
// Joins the parts of the rows whose keys were read in more than one, (m, l) and
// line of each: sum_s 2^(m_s - m) y_s over the same sum of l_s.
//
// Rows of sequences that the few-rows kernel takes (FEW): row r of a call of
// which it takes all, or else row r % (kFewRows KVH) of sequence r / (kFewRows
// KVH), of which it has kFewRows rows a head at most.
struct Parts {
    int64_t row;
    int n;                    // <= kMaxParts
    const float4 *lines;      // of part 0; `pitch` rows on for the next
    const float2 *ml;
    int64_t pitch;
};
// The pieces of a row that the few-rows kernel has cut, within the workspace whatever
// it holds.
template <int D, class C>
__device__ __forceinline__ bool find_cut(const KvArgs<C> &a, int64_t row, Parts &p) {
    const int2 info = cut_info(a, D)[row];
    p.row = row;
    p.n = info.y;
    if (p.n < 2 || p.n > kMaxParts || info.x < 0 || info.x / kRows > a.slots - p.n)
        return false;                                           // written directly
    p.pitch = kRows;
    p.lines = reinterpret_cast<const float4 *>(a.cut) + (int64_t)info.x * (D / 4);
    p.ml = reinterpret_cast<const float2 *>(a.cut + (int64_t)a.slots * kRows * D) + info.x;
    return true;
}
template <int D, bool FEW, class C>
__device__ __forceinline__ bool find_parts(const KvArgs<C> &a, int64_t row, Parts &p) {
    const Kv8Seqs &sq = a.seqs;
    int b, t;
    if (FEW && !a.mixed) return find_cut<D>(a, row, p);
    if (FEW) {
        const int each = kFewRows * a.c.KVH;
        b = (int)(row / each);
        const int r = (int)(row - (int64_t)b * each), h = r / kFewRows;
        t = q_at(sq, b) + r % kFewRows / a.G;
        row = (int64_t)t * a.QH + h * a.G + r % kFewRows % a.G;
    } else {
        t = (int)(row / a.QH);
        b = find_seq(sq.B, t, [&](int i) { return (int64_t)q_at(sq, i); });
    }
    const int q0 = q_at(sq, b), q1 = q_at(sq, b + 1);
    if (t < q0 || t >= q1) return false;
    const int64_t rows = (int64_t)(q1 - q0) * a.G;
    if (FEW) return rows <= a.max_rows && find_cut<D>(a, row, p);
    if (rows <= a.min_rows) return false;
    const int64_t keys = min((int64_t)sq.lengths[b] - (q1 - t) + 1, key_capacity(a));
    const int64_t chunk = keys_of_part(a, sq.lengths[b]);
    if (keys <= chunk) return false;                            // written directly
    p.row = row;
    p.n = (int)((keys + chunk - 1) / chunk);                    // <= S
    p.pitch = (int64_t)sq.n_tok * a.QH;
    p.lines = reinterpret_cast<const float4 *>(a.part) + row * (D / 4);
    p.ml = reinterpret_cast<const float2 *>(a.part + (int64_t)a.S * p.pitch * D) + row;
    return true;
}
// What find_parts leaves to be looked at beside the parts' loads where the
// few-rows kernel takes all rows: whether row p.row is of a sequence (if it is not,
// what find_cut has read is of no meaning).  As a step of loads in front of theirs it
// took 1 us.
template <bool FEW, class C>
__device__ __forceinline__ bool of_sequence(const KvArgs<C> &a, const Parts &p) {
    if (!FEW || a.mixed) return true;
    const int t = (int)(p.row / a.QH);
    if (a.seqs.B == 1) return t >= q_at(a.seqs, 0) && t < q_at(a.seqs, 1);
    const SeqPlace in = find_place(a.seqs, t, [](int q, int) { return (int64_t)q; });
    return t >= in.q0 && t < in.q1;
}

// Up to kWaveParts parts: a wave to a row, four rows to a workgroup, no barrier.
// The whole call with 4 parts of 20 rows 8.1 us (8.6 with a workgroup to a row),
// with 16 parts 8.4 (8.9); 64 ragged sequences, 1280 rows, 42.3 (42.9).
constexpr int kWaveParts = 16;
template <bool BF16, int D, bool FEW, class C>
__global__ __launch_bounds__(kThreads) void kv_join_wave_kernel(KvArgs<C> a, int64_t rows) {
    constexpr int V = D / 64;                                   // values a lane
    const int lane = threadIdx.x & 63;
    const int64_t r = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Parts p;
    if (r >= rows || !find_parts<D, FEW>(a, r, p) || p.n > kWaveParts) return;
    const float *src = reinterpret_cast<const float *>(p.lines) + V * lane;
    // all loads in flight together, at clamped places
    constexpr int kFirst = kWaveParts / 4;
    float x[kWaveParts][V], y[V];
    auto load = [&](int s0, int s1) {
#pragma unroll
        for (int s = s0; s < s1; ++s)
#pragma unroll
            for (int e = 0; e < V; ++e) x[s][e] = src[min(s, p.n - 1) * p.pitch * D + e];
    };
    load(0, kFirst);
    if (p.n > kFirst) load(kFirst, kWaveParts);
    const float2 v = p.ml[min(lane, p.n - 1) * p.pitch];
    if (!of_sequence<FEW>(a, p)) return;
    const float m = group_max(lane < p.n ? v.x : -INFINITY, 16);          // -inf in lanes 16 on
    const float f = lane < p.n ? exp2_fast(v.x - (m == -INFINITY ? 0.0f : m)) : 0.0f;
    float l = lane < p.n ? v.y * f : 0.0f;
    l += dpp_f32<kDppXor1>(l);
    l += dpp_f32<kDppXor2>(l);
    l += dpp_f32<kDppHalfMirror>(l);
    l += dpp_f32<kDppMirror>(l);
    l = lane_value(l, 0);
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = 0.0f;
    auto add = [&](int s0, int s1) {
#pragma unroll
        for (int s = s0; s < s1; ++s)
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = __builtin_fmaf(x[s][e], lane_value(f, s), y[e]);   // f = 0 from n on
    };
    add(0, kFirst);
    if (p.n > kFirst) add(kFirst, kWaveParts);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int64_t at = p.row * D + V * lane;
    if (BF16) {
        uint16_t *o = static_cast<uint16_t *>(a.out) + at;
        if (V == 2)
            *reinterpret_cast<uint32_t *>(o) = bf16_round(y[0] * inv) | bf16_round(y[V - 1] * inv) << 16;
        else
            *o = (uint16_t)bf16_round(y[0] * inv);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) static_cast<float *>(a.out)[at + e] = y[e] * inv;
    }
}

// More: a workgroup to a row.  The parts' weights 2^(m_s - m) go to LDS first;
// then D / 4 threads read a part, 16 bytes each, so that the workgroup has 4
// THREADS / D parts in flight: 1024 threads for up to kJoinRows rows, or else
// 256 (128 parts of 20 rows: 11.4 us with 256 threads, 4.7 with 1024; 4 parts of
// 1280 rows 4.9 and 10.3).
constexpr int kJoinRows = 512;
template <bool BF16, int D, int THREADS, bool FEW, class C>
__global__ __launch_bounds__(THREADS) void kv_join_kernel(KvArgs<C> a) {
    constexpr int kWide = D / 4, kLines = THREADS / kWide, kJoinWaves = THREADS / 64;
    __shared__ float weight[kMaxParts > THREADS ? kMaxParts : THREADS];
    __shared__ float red[2][kJoinWaves];
    __shared__ float4 sum[kJoinWaves][kWide];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Parts p;
    if (!find_parts<D, FEW>(a, blockIdx.x, p)) return;
    const int parts = p.n;
    const int64_t row = p.row, pitch = p.pitch;
    const float4 *lines = p.lines;
    const float2 *ml = p.ml;
    // the first lines are under way while the weights are formed
    const int d = threadIdx.x % kWide, line = threadIdx.x / kWide;
    const float4 first = lines[min(line, parts - 1) * pitch * kWide + d];
    constexpr int kEach = (kMaxParts + THREADS - 1) / THREADS;
    float2 v[kEach];
    float mm = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int s = threadIdx.x + i * THREADS;
        v[i] = s < parts ? ml[s * pitch] : make_float2(-INFINITY, 0.0f);
        mm = fmaxf(mm, v[i].x);
    }
    if (!of_sequence<FEW>(a, p)) return;                        // uniform
    mm = group_max(mm, 64);
    if (lane == 0) red[0][wave] = mm;
    __syncthreads();
    mm = group_max(red[0][lane % kJoinWaves], kJoinWaves);
    const float base = mm == -INFINITY ? 0.0f : mm;
    float ll = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const float f = exp2_fast(v[i].x - base);
        weight[threadIdx.x + i * THREADS] = f;
        ll += v[i].y * f;
    }
    ll = quad_sum(ll);
    ll += dpp_f32<kDppXor1>(ll);
    ll += dpp_f32<kDppXor2>(ll);
    ll += dpp_f32<kDppHalfMirror>(ll);
    ll += dpp_f32<kDppMirror>(ll);
    if (lane == 0) red[1][wave] = ll;
    __syncthreads();
    float f = weight[line];
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (line < parts) y = make_float4(first.x * f, first.y * f, first.z * f, first.w * f);
#pragma unroll 4
    for (int s = line + kLines; s < parts; s += kLines) {
        const float4 x = lines[s * pitch * kWide + d];
        f = weight[s];
        y.x += x.x * f; y.y += x.y * f; y.z += x.z * f; y.w += x.w * f;
    }
    // lanes kWide apart have the same values
    for (int o = kWide; o < 64; o *= 2) {
        y.x += __shfl_xor(y.x, o); y.y += __shfl_xor(y.y, o);
        y.z += __shfl_xor(y.z, o); y.w += __shfl_xor(y.w, o);
    }
    if (lane < kWide) sum[wave][lane] = y;
    __syncthreads();
    if (threadIdx.x < kWide) {
        ll = 0.0f;
        y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kJoinWaves; ++w) {
            ll += red[1][w];
            const float4 x = sum[w][threadIdx.x];
            y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
        }
        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
        store4<BF16>(a.out, row * D + 4 * threadIdx.x, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    }
}

int64_t join_threads(int64_t rows, int64_t parts) {
    if (parts <= kWaveParts) return (rows + kWaves - 1) / kWaves * kThreads;
    return rows * (rows <= kJoinRows ? 1024 : 256);
}
template <bool BF16, int D, bool FEW, class C>
void join(const KvArgs<C> &a, int64_t rows, int64_t parts, hipStream_t s) {
    if (parts <= kWaveParts)
        hipLaunchKernelGGL((kv_join_wave_kernel<BF16, D, FEW, C>), dim3((unsigned)((rows + kWaves - 1) / kWaves)),
                           dim3(kThreads), 0, s, a, rows);
    else if (rows <= kJoinRows)
        hipLaunchKernelGGL((kv_join_kernel<BF16, D, 1024, FEW, C>), dim3((unsigned)rows), dim3(1024), 0, s, a);
    else
        hipLaunchKernelGGL((kv_join_kernel<BF16, D, 256, FEW, C>), dim3((unsigned)rows), dim3(256), 0, s, a);
}

// What a call launches, from its sizes alone.  Where the sequences bring many
// rows on average and there is much to do (16-row units times their steps with
// all lengths at their limit, and 2 for the start and end of each, above
// kManyWork), those that do go to the kernel for many rows; the other takes the
// rest, or else all.  A lone workgroup of many rows takes 2 us a tile of 64 keys,
// so with little work the few-rows kernel, cut to fill the GPU, is done first
// though it reads and converts a code 8 times as often.  In us, few and many
// rows, 8-bit cache, tokens on keys of each sequence, 5 heads of 4 with D = 128, bf16 and
// fp32, then 8 heads of 2 with D = 64, bf16, with its own work:
//   work   640  128 on 500          8.5  20.9    9.7  28.8     512   5.9  15.7
//         2880  128 on 4000        30.7  29.6   34.0  36.6    2304  19.5  22.5
//         3840  8 x 64 on 1000     30.7  34.2   33.5  48.9
//         4480  256 on 3000        39.4  33.0   41.8  42.2
//         4800  16 x 48 on 700     28.9  26.7   31.9  37.6
//         5760  16 x 16 on 4000    65.3  55.4   66.3  75.6
//         7500  1000 on 1000       29.3  33.7   33.6  48.6
//         7680  4 x 256 on 1000    48.2  35.8   50.2  51.1    6144  21.2  26.2
//        11520  512 on 4000        68.6  54.2   74.7  76.1    9216  28.0  36.1
//        15360  64 x 48 on 500     72.5  49.7   82.8  70.8   12288  31.6  34.9
//        17280  8 x 96 on 4000      100  93.8    110   128   13824  44.8  69.8
//        20320  128 on 32000        191   118    202   164   16256   127  68.8
//        30720  64 x 96 on 500      132  68.8    154   101   24576  53.3  47.4
//        92160  64 x 64 on 4000     491   281    578   440   73728   203   232
// The bound is that of bf16 rows of D = 128.  For fp32 rows, and for two heads of
// 64 on a key head, it is too low: calls above it may take up to 1.7 times as long as by the
// few-rows kernel.
//
// Many rows: as many parts of the keys as keep a workgroup on every CU, if that
// can save three steps; how many a sequence has, and of what keys, its length
// says on the device (parts behind its end exit at once).
//
// The form and whether there is a join at all go by max_blocks, as a launch's grid
// has to: with room for 8192 keys 128 bf16 rows on 500 take 22.7 us and not 8.4, and one
// row on 200 takes 7.8 and not 6.0; on the 4-bit cache 512 rows on 512 25.3 and not 14.0,
// one row on 200 7.4 and not 5.5.
//
// Few rows: units are cut where one sequence may be longer than three steps and
// they are few, or where the longest could hold up the others or a prompt for
// long (kLongSteps: 54 us); otherwise the join would cost more than it saves.
struct Plan {
    bool many, few, cuts;
    int64_t steps;            // of the longest sequence that max_blocks allows
    int S;
    int64_t groups;           // of the few-rows kernel
    int most, slots, step_shift;
    int64_t part, cut;        // floats of the workspace
};
// What differs between the caches' formats.
struct Rules {
    double many_work;         // above which rows go to the kernel for many
    int many_groups;          // workgroups of that kernel to aim at with parts of the keys
    int one_seq_units;        // units of a single sequence above which pieces are for kGroups workgroups
    int lone_steps;           // steps up to which a single sequence that can fill the GPU is not cut
};
Plan plan_for(int64_t n_tok, int64_t QH, int64_t B, int64_t max_blocks, int64_t KVH, int64_t T, int64_t D,
              const Rules &rules) {
    const int64_t G = QH / KVH, keys = max_blocks * T, unit = kTile * kWaves;
    const int64_t steps = keys > 0 ? (keys + unit - 1) / unit : 1;
    const int64_t seqs = n_tok < B ? n_tok : B;
    Plan p = {};
    p.steps = steps;
    p.S = 1;
    p.many = n_tok * G > kFewRows * B && (double)n_tok * QH / kRows * (steps + 2) > rules.many_work;
    p.few = !p.many || B > 1;
    if (p.many) {
        const double tiles = n_tok * (double)G / kManyRows;
        int64_t parts = (int64_t)(rules.many_groups / (KVH * (tiles > seqs ? tiles : seqs)));
        parts = parts < 1 ? 1 : parts < steps ? parts : steps;
        if (steps - (steps + parts - 1) / parts >= 3) p.S = (int)parts;
        if (p.S > 1) p.part = (p.S * n_tok * QH * (D + 2) + 3) / 4 * 4;
    }
    if (p.few) {
        int64_t tiles = n_tok * G / kRows + seqs;
        if (p.many && tiles > seqs * kFewTiles) tiles = seqs * kFewTiles;
        const int64_t units = tiles * KVH;
        // one sequence: 32768 keys of 5 heads 19.6 us with 512, 16.5 with 256
        p.most = seqs == 1 && units <= rules.one_seq_units ? kCUs : kGroups;
        // longer steps where their number would pass 32 bits (units of kLineSeqs
        // sequences do not: n_tok QH / 16 + 256 KVH < 2^28)
        p.step_shift = kStepShift;
        auto line = [&] { return units * (((steps - 1) >> (p.step_shift - kStepShift)) + 1); };
        while (B <= kLineSeqs && line() >= (int64_t)1 << 30) ++p.step_shift;
        p.cuts = steps > 3 && B <= kLineSeqs &&
                 ((3 * KVH * seqs < 2 * p.most && (!p.many || p.S > 1)) || steps >= kLongSteps);
        // A single sequence with a unit for every workgroup is not cut (steps_of_piece), and
        // the join that finds nothing takes 3 us.  But q_start may name fewer rows than the
        // call has, as in a captured one: a token in it then waits for its steps one after
        // the other, so only where they are few.  4-bit cache, fp32, 1000 rows, joined and not:
        // all of them on 1777 keys of 5 heads of 4 52.3 and 48.7 us, of 8 heads of 2, D = 64,
        // 32.3 and 29.4; one token 9.0 and 15.1, 8.0 and 12.3 (on 4000 keys 9.4 and 28.1).
        if (B == 1 && steps <= rules.lone_steps && (n_tok * G + kRows - 1) / kRows * KVH >= p.most) p.cuts = false;
        p.groups = units;
        if (B > kLineSeqs) p.groups = (p.many ? B * kFewTiles : n_tok * G / kRows + B) * KVH;
        if (p.cuts) {
            p.groups = units + p.most;
            if (p.groups > line()) p.groups = line();
            p.slots = (int)(line() < 2 * p.most ? line() : 2 * p.most);
            p.cut = (int64_t)p.slots * kRows * (D + 2) + 2 * n_tok * QH;
        }
    }
    return p;
}

// The kernels of a cache's format.
template <class C>
struct Kernels {
    void (*few)(KvArgs<C>);
    void (*many)(KvArgs<C>);
    void (*mixed)(KvArgs<C>);
};
template <bool BF16, int D, class C>
hipError_t attend(KvArgs<C> a, const Plan &p, const Kernels<C> &k, hipStream_t s) {
    const int64_t rows = (int64_t)a.seqs.n_tok * a.QH;
    const dim3 block(kThreads);
    a.mixed = p.many && p.few;
    a.min_rows = a.mixed ? kFewRows : 0;
    a.max_rows = a.mixed ? kFewRows : rows;
    if (p.many) a.many_groups = ((int64_t)a.seqs.n_tok * a.G / kManyRows + a.seqs.B) * a.c.KVH;
    const int64_t groups = a.many_groups * p.S + p.groups;
    const int64_t join_rows = a.mixed ? (int64_t)a.seqs.B * kFewRows * a.c.KVH : rows;
    // all launches or none
    constexpr int64_t kMost = (int64_t)1 << 32;
    if (groups * kThreads >= kMost || (p.many && p.S > 1 && join_threads(rows, p.S) >= kMost) ||
        (p.cuts && join_threads(join_rows, p.steps) >= kMost))
        return hipErrorInvalidConfiguration;
    if (a.mixed)
        hipLaunchKernelGGL(k.mixed, dim3((unsigned)groups), block, 0, s, a);
    else if (p.many)
        hipLaunchKernelGGL(k.many, dim3((unsigned)a.many_groups, 1, (unsigned)p.S), block, 0, s, a);
    else
        hipLaunchKernelGGL(k.few, dim3((unsigned)groups), block, 0, s, a);
    if (p.many && p.S > 1) join<BF16, D, false>(a, rows, p.S, s);
    if (p.cuts) join<BF16, D, true>(a, join_rows, p.steps, s);
    return hipGetLastError();
}

template <class C>
KvArgs<C> kv_args(const Plan &p, const void *q, int QH, const Kv8Seqs &seqs, const C &cache, float scale,
                  void *out, float *ws) {
    KvArgs<C> a = {};
    a.q = q;
    a.out = out;
    a.seqs = seqs;
    a.c = cache;
    a.QH = QH;
    a.G = QH / a.c.KVH;
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    a.part = ws;
    a.S = p.S;
    a.cut = ws + p.part;
    a.cuts = p.cuts;
    a.most = p.most;
    a.slots = p.slots;
    a.step_shift = p.step_shift;
    return a;
}

}  // namespace
}  // namespace bl
