// kv8_attention.hip -- causal attention over the 8-bit key/value cache.
//
// out = sum_j p_j v_j / sum_j p_j, p_j = 2^(s_j - m), s_j = scale log2(e)
// q.k_j, m the running maximum: one pass over the keys, the sums rescaled by
// 2^(m_old - m) when the maximum grows.
//
// Both products run on fp16 matrix instructions with fp32 sums, 16x16x32 for few
// rows and 32x32x16 for many.
// An int8 code is exact in fp16: the byte with its sign bit flipped, put
// below the byte 0x64, reads as 1024 + (code + 128), and one packed add of
// -1152 leaves the code (v_xor per 4 codes, v_perm and v_pk_add_f16 per 2).
// The other operand is scaled by a power of two into fp16's range and, for
// fp32 rows, split into two halves of 11 bits each (two matrix instructions):
//   q      by row, its largest |q| to [2^13, 2^14);
//   p sv   the value scale goes with the weight, by u, a power of two >= every
//          value scale seen so far: p sv / u * 2^14 <= 2^14.
// bf16 rows keep q exactly and round p sv to 11 bits once: their result is
// rounded to 8.
//
// Rows of a tile: the query heads of one key/value head are neighbouring rows
// of one product, so a cached byte is read once for all of them: row r of
// sequence b is token r / G, head r % G (G query heads to a key head).
//
// Operand layouts for few rows (lane = 16 quad + low): S^T = K Q^T puts key 4 quad + i, row
// low into accumulator i.  Which key a row of the K operand is, is free: row 4
// g + i of the operand for keys tt holds key 16 g + 4 tt + i of the tile, so
// that lane quad g ends up with keys 16 g .. 16 g + 15 of its row -- exactly the
// P^T operand of O^T = V^T P^T, whose V^T operand is then 16 consecutive bytes
// of a row of the transposed V.  No value crosses lanes between the products.
// A quad's 16 tokens lie in one block of the cache whatever T is.
#include "kv8_common.h"

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

// Four int8 codes -> four fp16.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t v = w ^ 0x80808080u;
    const half2 bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    lo = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, perm(0x64646464u, v, 0x04010400u)) + bias);
    hi = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, perm(0x64646464u, v, 0x04030402u)) + bias);
}
__device__ __forceinline__ half8 codes8(uint32_t w0, uint32_t w1) {
    uint4 o;
    codes_to_f16(w0, o.x, o.y);
    codes_to_f16(w1, o.z, o.w);
    return __builtin_bit_cast(half8, o);
}

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

// Scores s (16 keys of a granule in 8 n accumulators: N = 2 of rows16, 1 of 8)
// to fp16 weights times w_sv: hi, and lo for fp32 rows; their sum into l.  For
// bf16 rows w_sv goes into the exponent (to half a step of base, 2^-14 at most,
// against the 2^-12 of the rounding): one multiply-add and one exponential a score.
template <bool BF16, int N, typename S>
__device__ __forceinline__ void weights(const S &s, float cs, float base, float w_sv, float &l, half8 *hi,
                                        half8 *lo) {
    const float w = fmaxf(w_sv, 1.4551915e-11f);          // 2^-36: below fp16's smallest step of kUnit
    const float shift = BF16 ? __builtin_amdgcn_logf(w) - base : -base;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint32_t h[4], z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float p0 = exp2_fast(__builtin_fmaf(s(8 * k + 2 * e), cs, shift));
            const float p1 = exp2_fast(__builtin_fmaf(s(8 * k + 2 * e + 1), cs, shift));
            sum += p0 + p1;
            const float y0 = BF16 ? p0 : p0 * w_sv, y1 = BF16 ? p1 : p1 * w_sv;
            h[e] = f16_pair(y0, y1);
            if (!BF16) z[e] = f16_rest(y0, y1, h[e]);
        }
        hi[k] = __builtin_bit_cast(half8, make_uint4(h[0], h[1], h[2], h[3]));
        if (!BF16) lo[k] = __builtin_bit_cast(half8, make_uint4(z[0], z[1], z[2], z[3]));
    }
    l = BF16 ? __builtin_fmaf(sum, __builtin_amdgcn_rcpf(w), l) : l + sum;
}

// A count of keys taken into [0, most].
__device__ __forceinline__ uint32_t keys_within(int64_t keys, uint32_t most) {
    return (uint32_t)min(max(keys, (int64_t)0), (int64_t)most);
}

struct Args {
    const void *q;
    void *out;
    Kv8Seqs seqs;
    Kv8Cache c;
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

__device__ __forceinline__ int64_t key_capacity(const Args &a) {
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
__device__ __forceinline__ int2 *cut_info(const Args &a, int D) {
    return reinterpret_cast<int2 *>(a.cut + (int64_t)a.slots * kRows * (D + 2));
}
__device__ __forceinline__ uint32_t steps_of(const Args &a, int length, int shift) {
    const int64_t keys = min(max((int64_t)length, (int64_t)1), max(key_capacity(a), (int64_t)1));
    return (uint32_t)((keys - 1) >> shift) + 1;
}
struct SeqWork {
    int q0, n, length;
    uint32_t tiles, steps;
};
__device__ __forceinline__ SeqWork work_of(const Args &a, int q0, int q1, int length) {
    SeqWork w;
    w.q0 = min(max(q0, 0), a.seqs.n_tok);
    w.n = min(max(q1, 0), a.seqs.n_tok) - w.q0;
    w.length = length;
    const int64_t rows = (int64_t)w.n * a.G;
    w.tiles = rows > 0 && rows <= a.max_rows ? (uint32_t)(rows + kRows - 1) / kRows : 0u;
    w.steps = steps_of(a, length, a.step_shift);
    return w;
}
__device__ __forceinline__ SeqWork work_of(const Args &a, int b) {
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

__device__ __forceinline__ uint32_t steps_of_piece(const Args &a, uint32_t units, uint32_t steps, uint32_t top) {
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
__device__ __forceinline__ bool find_unit(const Args &a, uint32_t pos, Piece &p) {
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
__device__ __forceinline__ bool find_piece(const Args &a, uint32_t pos, Piece &p) {
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
    p.h = p.work.tiles == 1 ? unit : unit / p.work.tiles;
    p.tile = unit - p.h * p.work.tiles;
    p.slot = p.pieces == 1 ? -1 : (int)(cut_before + unit * p.pieces);
    return true;
}

// Few rows: one workgroup to a piece; its waves take 64-key tiles in turn, each
// with sums of its own, joined in LDS.  The products' operands go from memory to
// registers, no LDS in the loop: a cached byte has one reader.  The next tile's
// K is under way from the moment this one's has been used, and so is V.
//
// Bound by memory where the sequences are alike (64 of 4096 keys, 335 MB: 72 us,
// 4.65 TB/s, a copy 4.78), else by the longest pieces: a lone wave takes 1.6 us
// of instructions for a 64-key tile, and while others load, 2.9 us.  (64 ragged,
// 163 MB: 36.4 us, 4.5 TB/s, and 4.2 the join.)  178 registers in bf16 with D =
// 128, two workgroups to a CU; a third, with q in LDS, took 79 us for 128
// sequences instead of 72.5.
template <int D>
struct FewLds {
    float join[kWaves][kRows][D + 4];
    float m[kWaves][kRows], l[kWaves][kRows];
};
template <bool BF16, int D>
__device__ __forceinline__ void few_rows(const Args &a, uint32_t group, FewLds<D> &lds) {
    constexpr int ND = D / 64;              // 64-value pieces of a row
    constexpr int NO = D / 16;              // 16-value tiles of the output
    constexpr int NS = BF16 ? 1 : 2;        // fp16 parts of q and of p sv
    auto &join = lds.join;
    auto &join_m = lds.m, &join_l = lds.l;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int low = lane & 15, quad = lane >> 4;
    const Kv8Seqs &sq = a.seqs;
    const Kv8Cache &c = a.c;
    const uint32_t G = (uint32_t)a.G;

    Piece piece;
    if (!(a.seqs.B <= kLineSeqs ? find_piece(a, group, piece) : find_unit(a, group, piece))) return;
    const int b = piece.b, q0 = piece.work.q0, n = piece.work.n;
    const int h = (int)piece.h;
    const uint32_t r0 = piece.tile * kRows;                       // of the sequence's n G < 2^31
    const int rows = (int)min((uint32_t)kRows, (uint32_t)n * G - r0);
    const int64_t start = (int64_t)piece.work.length - n;         // position of the first new token
    const int64_t end = min(start + (r0 + rows - 1) / G + 1, key_capacity(a));     // keys the tile sees
    const bool uncut = piece.pieces == 1;
    // key positions: below 2^31, and so are they with a few tiles more in 32 bits
    const uint32_t k0 = uncut ? 0 : piece.nth * piece.c << a.step_shift;
    const uint32_t k1 = keys_within(end, uncut ? 0x7FFFFFFFu : k0 + (piece.c << a.step_shift));
    const uint32_t slot = (uint32_t)piece.slot + piece.nth;       // of what is cut
    if (!uncut && slot >= (uint32_t)a.slots) return;              // starts that overlap

    // this lane's row (rows past the last repeat it; they are not written)
    const uint32_t r = r0 + min(low, rows - 1);
    const int tok = (int)(r / G);
    const int hq = h * G + (int)(r - tok * G);
    const int64_t row = (int64_t)(q0 + tok) * a.QH + hq;
    if (a.cuts && piece.nth == 0 && (int)threadIdx.x < rows)
        cut_info(a, D)[row] = make_int2(uncut ? -1 : piece.slot * kRows + low, (int)piece.pieces);
    const uint32_t sees = keys_within(start + tok + 1, k1);       // keys before this one

    // q of the row: values 64 dc + 16 quad + 8 half + 0..7 per matrix step
    half8 qh[NS][ND][2];
    float c_row;
    {
        float4 v[ND][4];
        float top = 0.0f;
#pragma unroll
        for (int dc = 0; dc < ND; ++dc)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[dc][e] = load4<BF16>(a.q, row * D + 64 * dc + 16 * quad + 4 * e);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(v[dc][e].x), fabsf(v[dc][e].y)),
                                       fmaxf(fabsf(v[dc][e].z), fabsf(v[dc][e].w))));
            }
        top = quad_max(top);
        const float f = a.scale2 < 0.0f ? -to_f16_range(top) : to_f16_range(top);
        c_row = a.scale2 / f;
#pragma unroll
        for (int dc = 0; dc < ND; ++dc)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t w[4], z[4];
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const float4 x = v[dc][2 * hf + e2];
                    const float x0 = x.x * f, x1 = x.y * f, x2 = x.z * f, x3 = x.w * f;
                    w[2 * e2] = f16_pair(x0, x1);
                    w[2 * e2 + 1] = f16_pair(x2, x3);
                    z[2 * e2] = f16_rest(x0, x1, w[2 * e2]);
                    z[2 * e2 + 1] = f16_rest(x2, x3, w[2 * e2 + 1]);
                }
                qh[0][dc][hf] = __builtin_bit_cast(half8, make_uint4(w[0], w[1], w[2], w[3]));
                if (NS == 2)
                    qh[NS - 1][dc][hf] = __builtin_bit_cast(half8, make_uint4(z[0], z[1], z[2], z[3]));
            }
    }

    float m = -INFINITY, above = -INFINITY, l = 0.0f, u = 0.0f, unit_u = 0.0f;      // unit_u = kUnit / u
    float4v o[NO];
#pragma unroll
    for (int i = 0; i < NO; ++i) o[i] = float4v{0.f, 0.f, 0.f, 0.f};

    const uint32_t first_tile = k0 + wave * kTile;
    constexpr uint32_t kStep = kWaves * kTile;
    const int32_t *table = sq.table + (int64_t)b * sq.max_blocks;
    // Block of this lane's quad of a tile: the table's entry is loaded a step
    // ahead, at a clamped place, and looked at only when it is used (a look at
    // once would wait for it, and for all loads before it, in every step); -1
    // where it holds no token.
    auto entry_at = [&](uint32_t tile) { return table[min(tile + 16 * quad, k1 - 1) >> c.t_shift]; };
    auto block_of = [&](uint32_t tile, int entry) {
        return tile + 16 * quad < k1 && entry >= 0 && entry < c.n_blocks ? entry : -1;
    };
    uint4 kb[4][ND], vb[NO];
    float sk = 0.0f, sv = 0.0f;
    auto load_k = [&](uint32_t tile, int id) {
        // this lane's operand row: key 16 g + 4 tt + i of the tile, 4 g + i = low
        const int g = low >> 2;
        const int idk = max(__shfl(id, 16 * g), 0);
        const int s0 = (int)((tile + 16 * g) & (c.T - 1)) + (low & 3);
        const int8_t *p = c.K + (((int64_t)idk * c.KVH + h) * c.T + s0) * D + 16 * quad;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int dc = 0; dc < ND; ++dc)
                kb[tt][dc] = *reinterpret_cast<const uint4 *>(p + 4 * tt * D + 64 * dc);
    };
    auto load_v = [&](uint32_t tile, int id) {
        const int64_t hb = (int64_t)max(id, 0) * c.KVH + h;
        sk = c.sk[hb];
        sv = c.sv[hb];
        const int8_t *p = c.V + (hb * D + low) * c.T + (int)((tile + 16 * quad) & (c.T - 1));
#pragma unroll
        for (int i = 0; i < NO; ++i)
            vb[i] = *reinterpret_cast<const uint4 *>(p + 16 * i * c.T);
    };

    if (first_tile < k1) {
        int id = block_of(first_tile, entry_at(first_tile));
        load_k(first_tile, id);
        int entry = entry_at(first_tile + kStep), id_next = -1;
        load_v(first_tile, id);
        for (uint32_t tile = first_tile; tile < k1; tile += kStep) {
            float4v s[4];
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                s[tt] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int dc = 0; dc < ND; ++dc) {
                    const half8 k_lo = codes8(kb[tt][dc].x, kb[tt][dc].y);
                    const half8 k_hi = codes8(kb[tt][dc].z, kb[tt][dc].w);
#pragma unroll
                    for (int x = 0; x < NS; ++x) {
                        s[tt] = mfma_16x16x32(k_lo, qh[x][dc][0], s[tt]);
                        s[tt] = mfma_16x16x32(k_hi, qh[x][dc][1], s[tt]);
                    }
                }
            }
            const uint32_t next = tile + kStep;
            const bool more = next < k1;
            if (more) {
                id_next = block_of(next, entry);
                load_k(next, id_next);
            }

            float cs = fmaxf(c_row * sk, kTiny);
            const uint32_t key0 = tile + 16 * quad;
            const bool whole = id >= 0 && key0 + 16 <= sees;
            // a scale that this row does not see is not to touch u, nor to meet a weight of 0
            const float sv_seen = id >= 0 && key0 < sees ? sv : 0.0f;
            if (__ballot(!whole) != 0) {
                const int lim = id >= 0 && key0 < sees ? (int)min(sees - key0, 16u) : 0;
#pragma unroll
                for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[tt][i] = 4 * tt + i < lim ? s[tt][i] : -INFINITY;
            }
            float top = s[0][0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e >> 2][e & 3]);
            top = quad_max(top * cs);
            const float u_new = fmaxf(u, pow2_above(quad_max(fabsf(sv_seen))));
            float base = m == -INFINITY ? 0.0f : m;
            if (__builtin_expect(__ballot(top > above || u_new != u) != 0, 0)) {
                const float m_new = fmaxf(m, top);
                float fix = m == -INFINITY ? 0.0f : exp2_fast(m - m_new);
                l *= fix;
                const float inverse = pow2_inverse(u_new);
                fix *= u * inverse;                        // u = 0 at first
                unit_u = kUnit * inverse;
#pragma unroll
                for (int i = 0; i < NO; ++i) o[i] *= fix;
                m = m_new;
                u = u_new;
                above = raise_above<BF16>(m);
                base = m == -INFINITY ? 0.0f : m;
                if (fabsf(base) >= kFarScore<BF16>) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e >> 2][e & 3] = s[e >> 2][e & 3] * cs - base;
                    cs = 1.0f;
                    base = 0.0f;
                }
            }
            half8 ph[NS][2];
            weights<BF16, 2>([&](int e) { return s[e >> 2][e & 3]; }, cs, base,
                             sv_seen * unit_u, l, ph[0], ph[NS - 1]);
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                const half8 v_lo = codes8(vb[i].x, vb[i].y), v_hi = codes8(vb[i].z, vb[i].w);
#pragma unroll
                for (int x = 0; x < NS; ++x) {
                    o[i] = mfma_16x16x32(v_lo, ph[x][0], o[i]);
                    o[i] = mfma_16x16x32(v_hi, ph[x][1], o[i]);
                }
            }
            if (more) {
                id = id_next;
                entry = entry_at(next + kStep);            // before V: loads come back in order
                load_v(next, id);
            }
        }
    }
    l = quad_sum(l);

    // join the waves: thread (row, values) sums what each brings
    const float unit = u / kUnit;
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) join[wave][low][16 * i + 4 * quad + e] = o[i][e] * unit;
    if (quad == 0) {
        join_m[wave][low] = m;
        join_l[wave][low] = l;
    }
    __syncthreads();
    constexpr int kPieces = kRows * D / 4 / kThreads;
#pragma unroll
    for (int pc = 0; pc < kPieces; ++pc) {
        const int at = (pc * kThreads + (int)threadIdx.x) * 4;
        const int rr = at / D, d = at % D;
        if (rr >= rows) continue;
        float mm = join_m[0][rr];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, join_m[w][rr]);
        const float base = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = exp2_fast(join_m[w][rr] - base);
            const float4 x = *reinterpret_cast<const float4 *>(&join[w][rr][d]);
            ll += join_l[w][rr] * f;
            y.x += x.x * f; y.y += x.y * f; y.z += x.z * f; y.w += x.w * f;
        }
        const uint32_t rj = r0 + rr, tj = rj / G;
        const int64_t row_j = (int64_t)(q0 + (int)tj) * a.QH + h * G + (rj - tj * G);
        if (uncut) {
            const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
            store4<BF16>(a.out, row_j * D + d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        } else {
            *reinterpret_cast<float4 *>(a.cut + ((int64_t)slot * kRows + rr) * D + d) = y;
            if (d == 0) {
                float *ml = a.cut + (int64_t)a.slots * kRows * D + ((int64_t)slot * kRows + rr) * 2;
                ml[0] = mm;
                ml[1] = ll;
            }
        }
    }
}

// Many rows: one workgroup per (128 rows, key head, part of the keys), 32 rows
// a wave, 64 keys at a time.  The workgroup turns the codes of a tile into fp16
// once, in LDS, for all rows (16-row workgroups did it for each: four
// conversions per matrix step).  While tile t is used, t + 1 is turned into
// the other buffer and the codes of t + 2 are on their way.
//
// Bound by vector instructions, about 380 of a wave and tile beside its 32
// matrix instructions: 40 of them exponentials, logarithms and reciprocals at half
// the rate, 87 the conversion.  2 x 2048 ragged rows on 4096 keys, 5
// heads of 4, bf16, 92 GFLOP: 131 us, 700 TFLOP/s (a large bf16 matrix product
// 1145); fp32, with two matrix instructions for one, 199 us.
//
// Layouts (lane = 32 half + low): S^T = K Q^T puts key 8 (i / 4) + 4 half + i
// % 4 of the operand's rows, row low, into accumulator i.  Operand row r holds
// key r with its bits 2 and 3 swapped, so accumulators 8 s .. 8 s + 7 are keys
// 16 s + 8 half .. + 7: the P^T operand of step s.
//
// LDS: K [64][D] and V^T [D][64] in 16-byte pieces, piece p of line y at p ^ y
// (K, D = 128) or p ^ (y / 2) (lines of 128 bytes), so that 16 lanes reading
// one piece of 16 lines touch every bank once.
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
__device__ __forceinline__ int64_t keys_of_part(const Args &a, int length) {
    const uint32_t steps = steps_of(a, length, kStepShift), each = (steps + a.S - 1) / (uint32_t)a.S;
    return (int64_t)(steps - each < 3 ? steps : each) << kStepShift;
}
template <int D>
struct ManyLds {
    uint4 k[2 * kTile * D / 8], v[2 * kTile * D / 8];
};
template <bool BF16, int D>
__device__ __forceinline__ void many_rows(const Args &a, int64_t at, int split, ManyLds<D> &lds) {
    constexpr int NS = BF16 ? 1 : 2;
    constexpr int NQ = D / 16;              // steps of K Q^T
    constexpr int NO = D / 32;              // tiles of the output
    constexpr int kPieces = kTile * D / 16 / kThreads;      // 16-byte pieces of K and of V per thread
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, gt = threadIdx.x;
    const int low = lane & 31, half = lane >> 5;
    // Heads of one tile side by side, tiles that see most first.  Two
    // workgroups share a CU: where all start at once, the second of each is to
    // be the first's complement, so the order turns round after the first 256.
    const int64_t groups = a.many_groups;
    if (at >= kCUs && groups <= 2 * kCUs) at = groups - 1 - (at - kCUs);
    const int h = (int)(at % a.c.KVH);
    const int64_t slot = at / a.c.KVH;
    const Kv8Seqs &sq = a.seqs;
    const Kv8Cache &c = a.c;
    const int G = a.G;
    const int b = find_seq(sq.B, slot, [&](int i) {
        return (int64_t)q_at(sq, i) * G / kManyRows + i;
    });
    const int q0 = q_at(sq, b), n = q_at(sq, b + 1) - q0;
    int64_t nth = slot - ((int64_t)q0 * G / kManyRows + b);
    const int64_t all_rows = (int64_t)n * G;
    const int64_t tiles = (all_rows + kManyRows - 1) / kManyRows;
    if (nth < 0 || n <= 0 || nth >= tiles || all_rows <= a.min_rows) return;
    nth = tiles - 1 - nth;                  // the rows that see most first
    const int64_t r0 = nth * kManyRows;
    const int64_t start = (int64_t)sq.lengths[b] - n;
    const int64_t cap = key_capacity(a);
    const int64_t end = min(start + (min(r0 + kManyRows, all_rows) - 1) / G + 1, cap);
    const int64_t chunk = keys_of_part(a, sq.lengths[b]);
    if (split > 0 && split * chunk >= end) return;
    const uint32_t k0 = (uint32_t)(split * chunk), k1 = keys_within(min(end, split * chunk + chunk), 0x7FFFFFFFu);

    const int64_t rw = r0 + 32 * wave;      // the wave's first row
    const bool rows_here = rw < all_rows;
    const int64_t r = min(rw + low, all_rows - 1);
    const int tok = (int)(r / G);
    const int64_t row = (int64_t)(q0 + tok) * a.QH + h * G + (int)(r - (int64_t)tok * G);
    const int64_t pos = start + tok;
    // the keys before this one are seen by this row, the wave's first and last
    const uint32_t sees = keys_within(pos + 1, k1);
    const uint32_t sees_lo = keys_within(start + min(rw, all_rows - 1) / G + 1, k1);
    const uint32_t sees_hi = keys_within(start + min(rw + 31, all_rows - 1) / G + 1, k1);

    half8 qh[NS][NQ];
    float c_row;
    {
        float4 v[NQ][2];
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < NQ; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[s][e] = load4<BF16>(a.q, row * D + 16 * s + 8 * half + 4 * e);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(v[s][e].x), fabsf(v[s][e].y)),
                                       fmaxf(fabsf(v[s][e].z), fabsf(v[s][e].w))));
            }
        top = fmaxf(top, __shfl_xor(top, 32));
        const float f = a.scale2 < 0.0f ? -to_f16_range(top) : to_f16_range(top);
        c_row = a.scale2 / f;
#pragma unroll
        for (int s = 0; s < NQ; ++s) {
            uint32_t w[4], z[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x0 = v[s][e].x * f, x1 = v[s][e].y * f, x2 = v[s][e].z * f, x3 = v[s][e].w * f;
                w[2 * e] = f16_pair(x0, x1);
                w[2 * e + 1] = f16_pair(x2, x3);
                if (NS == 2) {
                    z[2 * e] = f16_rest(x0, x1, w[2 * e]);
                    z[2 * e + 1] = f16_rest(x2, x3, w[2 * e + 1]);
                }
            }
            qh[0][s] = __builtin_bit_cast(half8, make_uint4(w[0], w[1], w[2], w[3]));
            if (NS == 2) qh[NS - 1][s] = __builtin_bit_cast(half8, make_uint4(z[0], z[1], z[2], z[3]));
        }
    }

    // A tile starts at a multiple of 64, so a key's slot is its own low bits,
    // and the tile's in blocks of 128.
    const int32_t *table = sq.table + (int64_t)b * sq.max_blocks;
    auto entry_at = [&](uint32_t t) { return table[min(t, k1 - 1) >> c.t_shift]; };    // as above
    auto block_of = [&](uint32_t t, int entry) {
        return t < k1 && entry >= 0 && entry < c.n_blocks ? entry : -1;
    };
    const uint32_t block_bytes = (uint32_t)(c.KVH * c.T) * D;              // < 2^31
    const int pk = gt / (D / 16), pv = gt >> 2;             // key and value of piece 0; + 32, + 64 of piece 1
    const int8_t *kp = c.K + ((int64_t)h * c.T + (pk & (c.T - 1))) * D + 16 * (gt % (D / 16));
    const int8_t *vp = c.V + ((int64_t)h * D + pv) * c.T + (16 * gt & 48 & (c.T - 1));
    const int k_next = c.T > 32 ? 32 * D : 0, v_next = 64 * c.T;
    uint4 kr[kPieces], vr[kPieces];
    int k_entry[kPieces], v_entry;
    float sk = 0.0f, sv = 0.0f, sk_next, sv_next;           // of granule lane % 4: 16 tokens of a tile
    bool in_use = false, in_use_next;
    auto load_ids = [&](uint32_t tile) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) k_entry[i] = entry_at(tile + pk + 32 * i);
        v_entry = entry_at(tile + 16 * (gt & 3));
    };
    // what lies behind k1 is read from block 0
    auto load_tile = [&](uint32_t tile) {
        const int in = (int)tile & (c.T - 1), vid = block_of(tile + 16 * (gt & 3), v_entry);
        const int8_t *vb = vp + (uint64_t)(uint32_t)max(vid, 0) * block_bytes + in;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int kid = block_of(tile + pk + 32 * i, k_entry[i]);
            kr[i] = *reinterpret_cast<const uint4 *>(kp + (uint64_t)(uint32_t)max(kid, 0) * block_bytes +
                                                     (in * D + i * k_next));
            vr[i] = *reinterpret_cast<const uint4 *>(vb + i * v_next);
        }
        const int64_t gb = (int64_t)max(vid, 0) * c.KVH + h;
        sk_next = c.sk[gb];
        sv_next = c.sv[gb];
        in_use_next = vid >= 0;
    };
    // LDS bytes: K line of 2 D bytes, V^T line of 128; a piece's place is its
    // number's 16 bytes XOR the line's, so that pieces of one line are reached
    // by an XOR of the thread's address, and lines 32 apart by an offset
    auto k_at = [](int key, int piece) {
        return D == 128 ? key * 256 + ((piece ^ (key & 15)) << 4) : key * 128 + ((piece ^ ((key >> 1) & 7)) << 4);
    };
    auto v_at = [](int d, int piece) { return d * 128 + ((piece ^ ((d >> 1) & 7)) << 4); };
    char *const lds_k = reinterpret_cast<char *>(lds.k), *const lds_v = reinterpret_cast<char *>(lds.v);
    constexpr int kBuf = kTile * D * 2;                     // bytes of a tile of K or V
    const int k_put = k_at(pk, 2 * (gt % (D / 16))), v_put = v_at(pv, 2 * (gt & 3));
    auto to_lds = [&](int buf) {
        const int ka = k_put + buf * kBuf, va = v_put + buf * kBuf;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            *reinterpret_cast<uint4 *>(lds_k + ka + i * 64 * D) = __builtin_bit_cast(uint4, codes8(kr[i].x, kr[i].y));
            *reinterpret_cast<uint4 *>(lds_k + (ka ^ 16) + i * 64 * D) = __builtin_bit_cast(uint4, codes8(kr[i].z, kr[i].w));
            *reinterpret_cast<uint4 *>(lds_v + va + i * 64 * 128) = __builtin_bit_cast(uint4, codes8(vr[i].x, vr[i].y));
            *reinterpret_cast<uint4 *>(lds_v + (va ^ 16) + i * 64 * 128) = __builtin_bit_cast(uint4, codes8(vr[i].z, vr[i].w));
        }
    };

    float m = -INFINITY, above = -INFINITY, l = 0.0f, u = 0.0f, unit_u = 0.0f;      // unit_u = kUnit / u
    float16v o[NO];
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    // operand row low holds key low, bits 2 and 3 swapped, of 32
    const int k_get = k_at((low & 0x13) | (low & 4) << 1 | (low & 8) >> 1, half), v_get = v_at(low, half);

    if (k0 < k1) {
        load_ids(k0);
        load_tile(k0);
        sk = sk_next;
        sv = sv_next;
        in_use = in_use_next;
        load_ids(k0 + kTile);
        to_lds(0);
        load_tile(k0 + kTile);
        load_ids(k0 + 2 * kTile);
        __syncthreads();
    }
    int buf = 0;
    for (uint32_t tile = k0; tile < k1; tile += kTile, buf ^= 1) {
        const bool here = rows_here && tile < sees_hi;
        // opaque, or the loop would hold an address for each piece
        int ka = k_get + buf * kBuf, va = v_get + buf * kBuf;
        asm("" : "+v"(ka), "+v"(va));
        __builtin_amdgcn_s_setprio(1);            // the CU's other workgroup fills what this leaves
        // also where the wave's rows do not see the tile: one block to schedule
        float16v s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
        for (int st = 0; st < NQ; ++st)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const half8 k = *reinterpret_cast<const half8 *>(lds_k + (ka ^ 32 * st) + t * 64 * D);
#pragma unroll
                for (int x = 0; x < NS; ++x) s[t] = mfma_32x32x16(k, qh[x][st], s[t]);
            }
        to_lds(buf ^ 1);
        __builtin_amdgcn_s_setprio(0);
        float cs[4], w_sv[4], sv_top = 0.0f;
        bool valid = true;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const bool ok = lane_value(in_use ? 1.0f : 0.0f, g) != 0.0f;
            cs[g] = fmaxf(c_row * lane_value(sk, g), kTiny);
            w_sv[g] = ok ? lane_value(sv, g) : 0.0f;
            valid = valid && ok;
            sv_top = fmaxf(sv_top, fabsf(w_sv[g]));
        }
        const bool used = in_use;
        sk = sk_next;
        sv = sv_next;
        in_use = in_use_next;
        load_tile(tile + 2 * kTile);
        load_ids(tile + 3 * kTile);
        if (here) {
            if (!(valid && tile + kTile <= sees_lo)) {                  // uniform
                const int lim = tile < sees ? (int)min(sees - tile, (uint32_t)kTile) : 0;
                sv_top = 0.0f;                              // as above: of what the row sees
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int lim_g = lane_value(used ? 1.0f : 0.0f, g) != 0.0f ? lim - 16 * g - 8 * half : 0;
                    w_sv[g] = lim > 16 * g ? w_sv[g] : 0.0f;
                    sv_top = fmaxf(sv_top, fabsf(w_sv[g]));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s[g >> 1][8 * (g & 1) + e] = e < lim_g ? s[g >> 1][8 * (g & 1) + e] : -INFINITY;
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float t8 = s[g >> 1][8 * (g & 1)];
#pragma unroll
                for (int e = 1; e < 8; ++e) t8 = fmaxf(t8, s[g >> 1][8 * (g & 1) + e]);
                top = fmaxf(top, t8 * cs[g]);
            }
            top = half_max(top);
            const float u_new = fmaxf(u, pow2_above(sv_top));
            float base = m == -INFINITY ? 0.0f : m;
            if (__builtin_expect(__ballot(top > above || u_new != u) != 0, 0)) {
                const float m_new = fmaxf(m, top);
                float fix = m == -INFINITY ? 0.0f : exp2_fast(m - m_new);
                l *= fix;
                const float inverse = pow2_inverse(u_new);
                fix *= u * inverse;                        // u = 0 at first
                unit_u = kUnit * inverse;
#pragma unroll
                for (int i = 0; i < NO; ++i) o[i] *= fix;
                m = m_new;
                u = u_new;
                above = raise_above<BF16>(m);
                base = m == -INFINITY ? 0.0f : m;
                if (fabsf(base) >= kFarScore<BF16>) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            s[g >> 1][8 * (g & 1) + e] = s[g >> 1][8 * (g & 1) + e] * cs[g] - base;
                        cs[g] = 1.0f;
                    }
                    base = 0.0f;
                }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {                  // 16 keys
                half8 p_hi, p_lo;
                weights<BF16, 1>([&](int e) { return s[g >> 1][8 * (g & 1) + e]; }, cs[g], base,
                                 w_sv[g] * unit_u, l, &p_hi, &p_lo);
#pragma unroll
                for (int i = 0; i < NO; ++i) {
                    const half8 v = *reinterpret_cast<const half8 *>(lds_v + (va ^ 32 * g) + i * 32 * 128);
                    o[i] = mfma_32x32x16(v, p_hi, o[i]);
                    if (NS == 2) o[i] = mfma_32x32x16(v, p_lo, o[i]);
                }
            }
        }
        __syncthreads();
    }

    if (rw + low >= all_rows) return;
    l = l + __shfl_xor(l, 32);
    float f0 = u / kUnit;
    const bool direct = min(pos + 1, cap) <= chunk;
    if (direct) {
        if (split > 0) return;
        f0 = l > 0.0f ? f0 / l : 0.0f;
    }
    const int64_t all = (int64_t)sq.n_tok * a.QH;
    float *dst = a.part + ((int64_t)split * all + row) * D;
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            float y[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) y[x] = o[i][e + x] * f0;
            const int d = 32 * i + 2 * e + 4 * half;
            if (direct) store4<BF16>(a.out, row * D + d, make_float4(y[0], y[1], y[2], y[3]));
            else store4<false>(dst, d, make_float4(y[0], y[1], y[2], y[3]));
        }
    if (!direct && half == 0) {
        float *ml = a.part + (int64_t)a.S * all * D + ((int64_t)split * all + row) * 2;
        ml[0] = m;
        ml[1] = l;
    }
}

template <bool BF16, int D>
__global__ __launch_bounds__(kThreads, 2) void kv8_few_kernel(Args a) {
    __shared__ FewLds<D> lds;
    few_rows<BF16, D>(a, blockIdx.x, lds);
}
template <bool BF16, int D>
__global__ __launch_bounds__(kThreads, 2) void kv8_many_kernel(Args a) {
    __shared__ ManyLds<D> lds;
    many_rows<BF16, D>(a, blockIdx.x, blockIdx.z, lds);
}
// Both in one launch: many rows wait for instructions, few rows for memory, so
// are to share the CUs.  The workgroups for few rows stand behind the first kCUs
// of the others.  15 single tokens on 8000 keys each beside a prompt of 500: 63.2
// us as two launches, 48.9 so; on 2000 keys beside one of 2000 75.9 and 63.7; 2
// prompts of up to 2048 rows alone 133.5 and 130.7.
template <bool BF16, int D>
__global__ __launch_bounds__(kThreads, 2) void kv8_mixed_kernel(Args a) {
    __shared__ union {
        FewLds<D> few;
        ManyLds<D> many;
    } lds;
    const int64_t all = a.many_groups * a.S, first = min(all, (int64_t)kCUs);
    const int64_t few = gridDim.x - all, i = blockIdx.x;
    if (i >= first && i < first + few) {
        few_rows<BF16, D>(a, (uint32_t)(i - first), lds.few);
    } else {
        const int64_t at = i < first ? i : i - few;
        const int split = (int)(at / a.many_groups);
        many_rows<BF16, D>(a, at - split * a.many_groups, split, lds.many);
    }
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
template <int D, bool FEW>
__device__ __forceinline__ bool find_parts(const Args &a, int64_t row, Parts &p) {
    const Kv8Seqs &sq = a.seqs;
    int b, t;
    if (FEW && a.mixed) {
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
    p.row = row;
    if (FEW) {
        if (rows > a.max_rows) return false;
        const int2 info = cut_info(a, D)[row];
        p.n = info.y;
        if (p.n < 2 || p.n > kMaxParts || info.x < 0 || info.x / kRows > a.slots - p.n)
            return false;                                       // written directly
        p.pitch = kRows;
        p.lines = reinterpret_cast<const float4 *>(a.cut) + (int64_t)info.x * (D / 4);
        p.ml = reinterpret_cast<const float2 *>(a.cut + (int64_t)a.slots * kRows * D) + info.x;
    } else {
        if (rows <= a.min_rows) return false;
        const int64_t keys = min((int64_t)sq.lengths[b] - (q1 - t) + 1, key_capacity(a));
        const int64_t chunk = keys_of_part(a, sq.lengths[b]);
        if (keys <= chunk) return false;                        // written directly
        p.n = (int)((keys + chunk - 1) / chunk);                // <= S
        p.pitch = (int64_t)sq.n_tok * a.QH;
        p.lines = reinterpret_cast<const float4 *>(a.part) + row * (D / 4);
        p.ml = reinterpret_cast<const float2 *>(a.part + (int64_t)a.S * p.pitch * D) + row;
    }
    return true;
}

// Up to kWaveParts parts: a wave to a row, four rows to a workgroup, no barrier.
// The whole call with 4 parts of 20 rows 8.1 us (8.6 with a workgroup to a row),
// with 16 parts 8.4 (8.9); 64 ragged sequences, 1280 rows, 42.3 (42.9).
constexpr int kWaveParts = 16;
template <bool BF16, int D, bool FEW>
__global__ __launch_bounds__(kThreads) void kv8_join_wave_kernel(Args a, int64_t rows) {
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
template <bool BF16, int D, int THREADS, bool FEW>
__global__ __launch_bounds__(THREADS) void kv8_join_kernel(Args a) {
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
template <bool BF16, int D, bool FEW>
void join(const Args &a, int64_t rows, int64_t parts, hipStream_t s) {
    if (parts <= kWaveParts)
        hipLaunchKernelGGL((kv8_join_wave_kernel<BF16, D, FEW>), dim3((unsigned)((rows + kWaves - 1) / kWaves)),
                           dim3(kThreads), 0, s, a, rows);
    else if (rows <= kJoinRows)
        hipLaunchKernelGGL((kv8_join_kernel<BF16, D, 1024, FEW>), dim3((unsigned)rows), dim3(1024), 0, s, a);
    else
        hipLaunchKernelGGL((kv8_join_kernel<BF16, D, 256, FEW>), dim3((unsigned)rows), dim3(256), 0, s, a);
}

// What a call launches, from its sizes alone.  Where the sequences bring many
// rows on average and there is much to do (16-row units times their steps with
// all lengths at their limit, and 2 for the start and end of each, above
// kManyWork), those that do go to the kernel for many rows; the other takes the
// rest, or else all.  A lone workgroup of many rows takes 2 us a tile of 64 keys,
// so with little work the few-rows kernel, cut to fill the GPU, is done first
// though it reads and converts a code 8 times as often.  In us, few and many
// rows, 5 heads of 4, bf16 (not measured for other heads and fp32):
//   work   120  128 rows on 500 keys      7.5  18.9
//          720  128 on 4000                13    19
//         1920  4 x 256 on 1000          22.9  29.5
//         2880  512 on 4000 / 8 x 64     31.7  27.7 / 35.4 42.5
//         3840  64 x 48 on 500           25.6    28
//         4320  8 x 96 on 4000             37    46
//         5080  128 on 32000             41.2  41.7
//         5440  4 x 128 on 8000          58.6  45.6
//         7680  64 x 96 on 500           44.5  29.8
//        23000  64 x 64 on 4000           191   142
// and with 32 rows a sequence, 64 on 4000 (work 11500) 110 and 140.
//
// Many rows: as many parts of the keys as keep a workgroup on every CU, if that
// can save three steps; how many a sequence has, and of what keys, its length
// says on the device (parts behind its end exit at once).
//
// The form and whether there is a join at all go by max_blocks, as a launch's grid
// has to: with room for 8192 keys 128 rows on 500 take 22 us and not 8, and one
// row on 200 takes 7.9 and not 5.8.
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
Plan plan_for(int64_t n_tok, int64_t QH, int64_t B, int64_t max_blocks, int64_t KVH, int64_t T, int64_t D) {
    const int64_t G = QH / KVH, keys = max_blocks * T, unit = kTile * kWaves;
    const int64_t steps = keys > 0 ? (keys + unit - 1) / unit : 1;
    const int64_t seqs = n_tok < B ? n_tok : B;
    Plan p = {};
    p.steps = steps;
    p.S = 1;
    p.many = n_tok * G > kFewRows * B && (double)n_tok * QH / kRows * (steps + 2) > kManyWork;
    p.few = !p.many || B > 1;
    if (p.many) {
        const double tiles = n_tok * (double)G / kManyRows;
        int64_t parts = (int64_t)(kCUs / (KVH * (tiles > seqs ? tiles : seqs)));
        parts = parts < 1 ? 1 : parts < steps ? parts : steps;
        if (steps - (steps + parts - 1) / parts >= 3) p.S = (int)parts;
        if (p.S > 1) p.part = (p.S * n_tok * QH * (D + 2) + 3) / 4 * 4;
    }
    if (p.few) {
        // one sequence: 32768 keys of 5 heads 19.6 us with 512, 16.5 with 256
        p.most = seqs == 1 ? kCUs : kGroups;
        int64_t tiles = n_tok * G / kRows + seqs;
        if (p.many && tiles > seqs * kFewTiles) tiles = seqs * kFewTiles;
        const int64_t units = tiles * KVH;
        // longer steps where their number would pass 32 bits (units of kLineSeqs
        // sequences do not: n_tok QH / 16 + 256 KVH < 2^28)
        p.step_shift = kStepShift;
        auto line = [&] { return units * (((steps - 1) >> (p.step_shift - kStepShift)) + 1); };
        while (B <= kLineSeqs && line() >= (int64_t)1 << 30) ++p.step_shift;
        p.cuts = steps > 3 && B <= kLineSeqs &&
                 ((3 * KVH * seqs < 2 * p.most && (!p.many || p.S > 1)) || steps >= kLongSteps);
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

template <bool BF16, int D>
hipError_t attend(Args a, const Plan &p, hipStream_t s) {
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
        hipLaunchKernelGGL((kv8_mixed_kernel<BF16, D>), dim3((unsigned)groups), block, 0, s, a);
    else if (p.many)
        hipLaunchKernelGGL((kv8_many_kernel<BF16, D>), dim3((unsigned)a.many_groups, 1, (unsigned)p.S), block, 0, s, a);
    else
        hipLaunchKernelGGL((kv8_few_kernel<BF16, D>), dim3((unsigned)groups), block, 0, s, a);
    if (p.many && p.S > 1) join<BF16, D, false>(a, rows, p.S, s);
    if (p.cuts) join<BF16, D, true>(a, join_rows, p.steps, s);
    return hipGetLastError();
}

}  // namespace

size_t kv8_attention_ws_floats(int64_t n_tok, int64_t QH, int64_t B, int64_t max_blocks,
                               int64_t KVH, int64_t T, int64_t D) {
    const Plan p = plan_for(n_tok, QH, B, max_blocks, KVH, T, D);
    return (size_t)(p.part + p.cut);
}

hipError_t launch_kv8_attention(const void *q, int dtype, int QH, const Kv8Seqs &seqs,
                                const bl_kv8 &cache, float scale, void *out, float *ws,
                                hipStream_t s) {
    const Plan p = plan_for(seqs.n_tok, QH, seqs.B, seqs.max_blocks, cache.KVH, cache.T, cache.D);
    Args a = {};
    a.q = q;
    a.out = out;
    a.seqs = seqs;
    a.c = kv8_device(cache);
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
    if (cache.D == 64) return dtype ? attend<true, 64>(a, p, s) : attend<false, 64>(a, p, s);
    return dtype ? attend<true, 128>(a, p, s) : attend<false, 128>(a, p, s);
}

}  // namespace bl
