// kv4_attention.hip -- causal attention over the 4-bit key/value cache.
//
// With a key z_j + s_j u_j and a value z'_j + s'_j u'_j (u, u' codes 0 .. 15):
//   x_j = scale log2(e) q.k_j = s_j (c q.u_j) + z_j (c sum q),  c = scale log2(e)
//   out = (sum_j p_j s'_j u'_j + sum_j p_j z'_j) / sum_j p_j,  p_j = 2^(x_j - r)
// over one pass of the keys, r following the running maximum of x.  The products
// q.u and sum (p s') u' run on fp16 matrix instructions with fp32 sums; a token's
// z and s meet its score and its weight in fp32, straight from their fp16 halves
// (v_fma_mix), so that no code is rounded.
//
// A code as fp16.  The nibble put below 0x64 (0x54 where it stands four bits
// higher) reads as 1024 + u (64 + u), and one packed add leaves u, or u - 8.  fp32
// rows take u - 8 with z + 8 s in z's place: with u itself the two sums of a
// result cancel (8 steps against what is left of a mean over many values), and
// errors of 1e-6 became 3e-6.  bf16 rows of the few-rows kernel take the nibble as it is, fp16's u 2^-24 or u
// 2^-20 (matrix instructions keep subnormals): two operations fewer of nine for
// eight codes; the other operand's odd pairs are 2^-4 instead.  Eight codes of a
// dword come out as the pairs (0, 4) (1, 5) (2, 6) (3, 7): a product's order of
// terms is free, so q and the weights are put into that order.
//
// The other operand is scaled by a power of two into fp16's range and, for fp32
// rows, split into two halves of 11 bits each (two matrix instructions):
//   q      by row, its largest |q| to [2^13, 2^14);
//   p s'   r = max x + log2(u) - 14 with u a power of two above every s' that the
//          row has seen: p s' <= 2^14, whatever the steps.
// bf16 rows keep q exactly and round p s' to 11 bits once: their result is
// rounded to 8.
//
// Layouts for few rows (lane = 16 quad + low) as for the 8-bit cache: S^T = K Q^T
// puts key 4 quad + i, row low into accumulator i, row 4 g + i of the K operand
// for keys tt holds key 16 g + 4 tt + i, so that a quad ends up with 16
// neighbouring keys of its row, which is the P^T operand of O^T = V^T P^T.  Row
// `low` of the V^T operand's tiles 2 i and 2 i + 1 is value 32 i + 2 low and the
// next, 16 bytes of the cache's 16-token group.
#include "kv4_common.h"
#include "kv_attention.h"

namespace bl {
namespace {

using Args = KvArgs<Kv4Cache>;

// (w & mask) | base in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t base) {
    uint32_t o;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(o) : "v"(w), "s"(mask), "v"(base));
    return o;
}
// Eight codes u -> fp16 u - CENTRE, pairs (0, 4) (1, 5) (2, 6) (3, 7).
template <int CENTRE>
__device__ __forceinline__ half8 codes8(uint32_t w) {
    const half2 b0 = {(_Float16)(-1024.0f - CENTRE), (_Float16)(-1024.0f - CENTRE)};
    const half2 b1 = {(_Float16)(-64.0f - CENTRE), (_Float16)(-64.0f - CENTRE)};
    const uint32_t v = w >> 8;
    uint4 o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, and_or(w, 0x000F000Fu, 0x64006400u)) + b0);
    o.y = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, and_or(w, 0x00F000F0u, 0x54005400u)) + b1);
    o.z = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, and_or(v, 0x000F000Fu, 0x64006400u)) + b0);
    o.w = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, and_or(v, 0x00F000F0u, 0x54005400u)) + b1);
    return __builtin_bit_cast(half8, o);
}
// The same pairs as they stand: u 2^-24 and, the odd ones, u 2^-20.
__device__ __forceinline__ half8 codes8_raw(uint32_t w) {
    const uint32_t v = w >> 8;
    return __builtin_bit_cast(half8, make_uint4(w & 0x000F000Fu, w & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u));
}
constexpr float kRaw = 16777216.0f;         // 2^24
// A pair of the other operand times 2^-4.
__device__ __forceinline__ uint32_t sixteenth(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, w) * half2{(_Float16)0.0625f, (_Float16)0.0625f});
}

// What fp16 leaves of a pair that was rounded to `h`; `minus` is -1 in a register,
// so that each half is one mixed multiply-add.
__device__ __forceinline__ uint32_t rest_of(float a, float b, uint32_t h, float minus) {
    const half2 v = __builtin_bit_cast(half2, h);
    const half2 r = {(_Float16)__builtin_fmaf((float)v[0], minus, a), (_Float16)__builtin_fmaf((float)v[1], minus, b)};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float minus_one() {
    float m = -1.0f;
    asm("" : "+s"(m));
    return m;
}
// z + 8 s.
__device__ __forceinline__ float middle(uint32_t zs) {
    return __builtin_fmaf((float)zs_s(zs), 8.0f, (float)zs_z(zs));
}

// A power of two above a step (0 <= s < 2^16), 2^-24 at least.
__device__ __forceinline__ float step_above(float s) {
    return __uint_as_float(max((__float_as_uint(s) & 0x7F800000u) + 0x00800000u, 103u << 23));
}
// log2 of a power of two.
__device__ __forceinline__ float log2_of(float u) { return (float)((int)(__float_as_uint(u) >> 23) - 127); }

constexpr float kUnitBits = 14.0f;

// What the sums of a row refer to: 2^(r1 + r2).  r1 = max + log2(u) - 14 and r2 = 0
// while that is exact enough, r1 = max and r2 = log2(u) - 14 for scores far from
// zero, from which r1 is taken before r2 (as for the 8-bit cache, see
// kFarScore).
struct Reference {
    float m = -INFINITY, above = -INFINITY, u = 0.0f, r1 = 0.0f, r2 = 0.0f;
    bool far = false;
    // To a maximum `top` and steps below u_new; what the sums are to be multiplied by.
    __device__ __forceinline__ float follow(float top, float u_new) {
        const bool none = m == -INFINITY;
        m = fmaxf(m, top);
        u = u_new;
        above = raise_above<false>(m);
        const float base = m == -INFINITY ? 0.0f : m, shift = log2_of(u) - kUnitBits;
        far = fabsf(base) >= kFarScore<false>;
        const float n1 = far ? base : base + shift, n2 = far ? shift : 0.0f;
        const float fix = none ? 0.0f : exp2_fast((r1 - n1) + (r2 - n2));
        r1 = n1;
        r2 = n2;
        return fix;
    }
};

// One workgroup to a piece; its waves take 64-key tiles in turn, each with sums of
// its own, joined in LDS.  Operands go from memory to registers, no LDS and no
// barrier in the loop: a cached byte has one reader.  The next tile's K is under way
// from the moment this one's has been used, and so is V.
//
// Single tokens wait for the chain starts -> entry -> K -> scores -> V, for memory, and for
// the join: 64 ragged sequences of up to 4096 keys, 5 heads of 4, bf16, 87 MB: 25.7 us, 3.4
// TB/s (the 8-bit cache's kernel reads 4.65 where all lengths are equal), 53% of a SIMD's
// time vector instructions, 37% of the waves' waiting, 1.4 waves of 2 on average; the whole
// call 27.7.  About 370 vector instructions a wave and
// tile (662 with one more add for each pair of codes, scores multiplied twice, and
// loads behind a branch, which copied every loaded register: 36.2 us).  Loads of V
// held in front of the loop's end: the same.  A third workgroup on a CU (168
// registers, 768 pieces): 25.2.  Units of 32 rows, which turn a code once for two
// products: 2048 bf16 rows on 4096 keys 135 us, of 16 rows 138 (124 with the tiles that see
// most first).
template <int D>
struct FewLds {
    float join[kWaves][kRows][D + 4];
    float m[kWaves][kRows], l[kWaves][kRows];
};
template <bool BF16, int D>
__device__ __forceinline__ void few_rows(const Args &a, uint32_t group, FewLds<D> &lds) {
    constexpr int NQ = D / 32;              // matrix steps of K Q^T, dwords of a lane's piece of a key
    constexpr int NO = D / 16;              // 16-value tiles of the output
    constexpr int NS = BF16 ? 1 : 2;        // fp16 parts of q and of p s
    auto &join = lds.join;
    auto &join_m = lds.m, &join_l = lds.l;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int low = lane & 15, quad = lane >> 4;
    const Kv8Seqs &sq = a.seqs;
    const Kv4Cache &c = a.c;
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

    const float minus = minus_one();
    // q of the row: values D / 4 quad + 8 j + 0 .. 7 for matrix step j
    half8 qh[NS][NQ];
    float c_row, q_sum = 0.0f;
    {
        float4 v[NQ][2];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 x = load4<BF16>(a.q, row * D + D / 4 * quad + 8 * j + 4 * e);
                v[j][e] = x;
                q_sum += (x.x + x.y) + (x.z + x.w);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
            }
        top = quad_max(top);
        const float f = a.scale2 < 0.0f ? -to_f16_range(top) : to_f16_range(top);
        q_sum = quad_sum(q_sum) * (BF16 ? f / kRaw : f);
        c_row = fmaxf(BF16 ? a.scale2 / f * kRaw : a.scale2 / f, kTiny);
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const float x[8] = {v[j][0].x * f, v[j][0].y * f, v[j][0].z * f, v[j][0].w * f,
                                v[j][1].x * f, v[j][1].y * f, v[j][1].z * f, v[j][1].w * f};
            uint32_t w[4], z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = f16_pair(x[e], x[e + 4]);
                if (!BF16) z[e] = rest_of(x[e], x[e + 4], w[e], minus);
                if (BF16 && (e & 1)) w[e] = sixteenth(w[e]);
            }
            qh[0][j] = __builtin_bit_cast(half8, make_uint4(w[0], w[1], w[2], w[3]));
            if (NS == 2) qh[NS - 1][j] = __builtin_bit_cast(half8, make_uint4(z[0], z[1], z[2], z[3]));
        }
    }

    Reference ref;
    float l = 0.0f, o_z = 0.0f;
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
    uint32_t kb[4][NQ];
    uint4 vb[NO / 2];
    uint32_t zk[16], zv[16];                // of the quad's 16 tokens
    auto load_zs = [&](uint32_t *zs, const uint32_t *from, uint32_t tile, int id) {
        const uint4 *p = reinterpret_cast<const uint4 *>(
            from + (((int64_t)max(id, 0) * c.KVH + h) << c.t_shift) + ((tile + 16 * quad) & (c.T - 1)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 w = p[i];
            zs[4 * i] = w.x;
            zs[4 * i + 1] = w.y;
            zs[4 * i + 2] = w.z;
            zs[4 * i + 3] = w.w;
        }
    };
    auto load_k = [&](uint32_t tile, int id) {
        // this lane's operand row: key 16 g + 4 tt + i of the tile, 4 g + i = low
        const int g = low >> 2;
        const int idk = max(__shfl(id, 16 * g), 0);
        const int s0 = (int)((tile + 16 * g) & (c.T - 1)) + (low & 3);
        const uint8_t *p = c.K + ((((int64_t)idk * c.KVH + h) << c.t_shift) + s0) * (D / 2) + D / 8 * quad;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
            if (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4 *>(p + 4 * tt * (D / 2));
                kb[tt][0] = w.x;
                kb[tt][1] = w.y;
                kb[tt][NQ - 2] = w.z;
                kb[tt][NQ - 1] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(p + 4 * tt * (D / 2));
                kb[tt][0] = w.x;
                kb[tt][1] = w.y;
            }
        }
        load_zs(zk, c.zk, tile, id);
    };
    auto load_v = [&](uint32_t tile, int id) {
        const int64_t g = (((int64_t)max(id, 0) * c.KVH + h) << (c.t_shift - 4)) + (((tile + 16 * quad) & (c.T - 1)) >> 4);
        const uint4 *p = reinterpret_cast<const uint4 *>(c.V + g * (8 * D)) + low;
#pragma unroll
        for (int i = 0; i < NO / 2; ++i) vb[i] = p[16 * i];
        load_zs(zv, c.zv, tile, id);
    };

    if (first_tile < k1) {
        int id = block_of(first_tile, entry_at(first_tile));
        load_k(first_tile, id);
        int entry = entry_at(first_tile + kStep), id_next = -1;
        load_v(first_tile, id);
        for (uint32_t tile = first_tile; tile < k1; tile += kStep) {
            float x[16];                    // scores of the quad's tokens over c_row
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                float4v s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const half8 k = BF16 ? codes8_raw(kb[tt][j]) : codes8<8>(kb[tt][j]);
#pragma unroll
                    for (int e = 0; e < NS; ++e) s = mfma_16x16x32(k, qh[e][j], s);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t zs = zk[4 * tt + i];
                    const float z_part = BF16 ? __builtin_fmaf(q_sum, (float)zs_z(zs), 0.0f) : q_sum * middle(zs);
                    x[4 * tt + i] = __builtin_fmaf(s[i], (float)zs_s(zs), z_part);
                }
            }
            // also behind the last tile (block 0's then): a branch would cost a copy of
            // every register that is loaded
            const uint32_t next = tile + kStep;
            id_next = block_of(next, entry);
            load_k(next, id_next);

            const uint32_t key0 = tile + 16 * quad;
            const bool whole = id >= 0 && key0 + 16 <= sees;
            if (__ballot(!whole) != 0) {
                // what stands in slots without a token may be anything, NaN too
                const int lim = id >= 0 && key0 < sees ? (int)min(sees - key0, 16u) : 0;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[e] = e < lim ? x[e] : -INFINITY;
                    zv[e] = e < lim ? zv[e] : 0u;
                }
            }
            float top = x[0];
            uint32_t zs_top = zv[0];                       // s is the upper half and not negative
#pragma unroll
            for (int e = 1; e < 16; ++e) {
                top = fmaxf(top, x[e]);
                zs_top = max(zs_top, zv[e]);
            }
            top = quad_max(top * c_row);
            const float u_new = fmaxf(ref.u, step_above(quad_max((float)zs_s(zs_top))));
            if (__builtin_expect(__ballot(top > ref.above || u_new != ref.u) != 0, 0)) {
                const float fix = ref.follow(top, u_new);
                l *= fix;
                o_z *= fix;
#pragma unroll
                for (int i = 0; i < NO; ++i) o[i] *= fix;
            }
            float base = ref.r1, cs = c_row;
            if (__ballot(ref.far) != 0) {                  // r2 is 0 for rows that are not
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = x[e] * c_row - ref.r1;
                base = ref.r2;
                cs = 1.0f;
            }
            half8 ph[NS][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t hi[4], lo[4];
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t zs = zv[8 * k + e];
                    const float p = exp2_fast(__builtin_fmaf(x[8 * k + e], cs, -base));
                    l += p;
                    o_z = __builtin_fmaf(p, BF16 ? (float)zs_z(zs) : middle(zs), o_z);
                    y[e] = __builtin_fmaf(p, (float)zs_s(zs), 0.0f);
                    if (!BF16) asm("" : "+v"(y[e]));       // formed once, for both halves
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hi[e] = f16_pair(y[e], y[e + 4]);
                    if (!BF16) lo[e] = rest_of(y[e], y[e + 4], hi[e], minus);
                    if (BF16 && (e & 1)) hi[e] = sixteenth(hi[e]);
                }
                ph[0][k] = __builtin_bit_cast(half8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                if (!BF16) ph[NS - 1][k] = __builtin_bit_cast(half8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
#pragma unroll
            for (int i = 0; i < NO / 2; ++i) {
                const half8 v00 = BF16 ? codes8_raw(vb[i].x) : codes8<8>(vb[i].x);
                const half8 v01 = BF16 ? codes8_raw(vb[i].y) : codes8<8>(vb[i].y);
                const half8 v10 = BF16 ? codes8_raw(vb[i].z) : codes8<8>(vb[i].z);
                const half8 v11 = BF16 ? codes8_raw(vb[i].w) : codes8<8>(vb[i].w);
#pragma unroll
                for (int e = 0; e < NS; ++e) {
                    o[2 * i] = mfma_16x16x32(v00, ph[e][0], o[2 * i]);
                    o[2 * i + 1] = mfma_16x16x32(v10, ph[e][0], o[2 * i + 1]);
                    o[2 * i] = mfma_16x16x32(v01, ph[e][1], o[2 * i]);
                    o[2 * i + 1] = mfma_16x16x32(v11, ph[e][1], o[2 * i + 1]);
                }
            }
            id = id_next;
            entry = entry_at(next + kStep);                // before V: loads come back in order
            load_v(next, id);
        }
    }
    // from 2^(r1 + r2) to 2^r1
    const float f_r2 = exp2_fast(ref.r2);
    l = quad_sum(l) * f_r2;
    o_z = quad_sum(o_z);

    // join the waves: thread (row, values) sums what each brings
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            join[wave][low][32 * (i / 2) + 2 * (4 * quad + e) + (i & 1)] = ((BF16 ? o[i][e] * kRaw : o[i][e]) + o_z) * f_r2;
    if (quad == 0) {
        join_m[wave][low] = ref.m == -INFINITY ? -INFINITY : ref.r1;
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

// Many bf16 rows: one workgroup per (128 rows, key head, part of the keys), 32 rows
// a wave, 64 keys at a time, the tile turned into fp16 once, in LDS, for all rows.  While
// tile t is used, t + 1 is turned into the other buffer and the codes of t + 2
// are on their way.  What goes to LDS are the keys and values themselves, fp16(z
// + s u), an error of 2^-11 at most beside the result's 2^-8: no z or s is left in the
// loop over scores.  (fp32 rows would need the codes and each token's z and s: 283 us
// for 2048 rows on 4096 keys, 5 heads of 4 and D = 128, where 16-row units take 181.)
//
// Bound by vector and matrix instructions that hardly overlap: 2 x 2048 ragged rows
// on 4096 keys, 5 heads of 4, 92 GFLOP: 133 us, 690 TFLOP/s (a large fp16 product
// 1420); of a SIMD's time 53% vector and 30% matrix instructions, 1.55 waves on
// average.  Scores of the next tile interleaved with this one's weights: 147; a
// raised priority for either part: the same.
//
// z and s that are not finite (never written by the append) count as 0 here, and
// a step with which a code of 15 would pass fp16 as the largest that does not:
// a token that rows do not see is in their products, times 0.
//
// Layouts (lane = 32 half + low): S^T = K Q^T puts key 8 (i / 4) + 4 half + i
// % 4 of the operand's rows, row low, into accumulator i.  Operand row r holds
// key r with its bits 2 and 3 swapped, so accumulators 8 s .. 8 s + 7 are keys
// 16 s + 8 half .. + 7: the P^T operand of step s.
//
// LDS: K [64][D] and V^T [D][64] in 16-byte pieces, piece p of line y at p ^ y
// (K, D = 128) or p ^ (y / 2) (lines of 128 bytes), so that 16 lanes reading
// one piece of 16 lines touch every bank once.
constexpr float kMostF16 = 65504.0f;

// A token's z and s as the tile takes them.
__device__ __forceinline__ uint32_t sound(uint32_t zs) {
    const float z = (float)zs_z(zs), s = (float)zs_s(zs);
    const bool fine = fabsf(z) <= kMostF16 && s >= 0.0f && s <= kMostF16;
    // less a half step of an 11-bit mantissa and its rounding: 15 s + z <= 65504
    const float most = (kMostF16 - z) * (0.99951172f / 15.0f);
    const half2 h = {(_Float16)z, (_Float16)fminf(s, most)};
    return fine ? __builtin_bit_cast(uint32_t, h) : 0u;
}
// Eight codes as the values z + s u, pairs as codes8; s and z by pair.
__device__ __forceinline__ half8 values8(uint32_t w, const uint32_t *s, const uint32_t *z) {
    const uint4 u = __builtin_bit_cast(uint4, codes8<0>(w));
    auto value = [&](uint32_t x, int i) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2, x),
                                                                      __builtin_bit_cast(half2, s[i]),
                                                                      __builtin_bit_cast(half2, z[i])));
    };
    return __builtin_bit_cast(half8, make_uint4(value(u.x, 0), value(u.y, 1), value(u.z, 2), value(u.w, 3)));
}

template <int D>
struct ManyLds {
    uint4 k[2 * kTile * D / 8], v[2 * kTile * D / 8];
    alignas(16) uint32_t held[2][kWaves];   // whether a granule holds tokens
    alignas(16) uint32_t pairs[kWaves][16]; // of a wave's 16 tokens of V, s and z by pair of codes8
};
template <int D>
__device__ __forceinline__ void many_rows(const Args &a, int64_t at, int split, ManyLds<D> &lds) {
    constexpr int NQ = D / 16;              // steps of K Q^T
    constexpr int NO = D / 32;              // tiles of the output
    constexpr int NW = D / 32;              // dwords of K's and of V's codes per thread
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
    const Kv4Cache &c = a.c;
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

    half8 qh[NQ];
    float c_row;
    {
        float4 v[NQ][2];
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < NQ; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 x = load4<true>(a.q, row * D + 16 * s + 8 * half + 4 * e);
                v[s][e] = x;
                top = fmaxf(top, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
            }
        top = half_max(top);
        const float f = a.scale2 < 0.0f ? -to_f16_range(top) : to_f16_range(top);
        c_row = fmaxf(a.scale2 / f, kTiny);
#pragma unroll
        for (int s = 0; s < NQ; ++s) {
            const float x[8] = {v[s][0].x * f, v[s][0].y * f, v[s][0].z * f, v[s][0].w * f,
                                v[s][1].x * f, v[s][1].y * f, v[s][1].z * f, v[s][1].w * f};
            qh[s] = __builtin_bit_cast(half8, make_uint4(f16_pair(x[0], x[4]), f16_pair(x[1], x[5]),
                                                         f16_pair(x[2], x[6]), f16_pair(x[3], x[7])));
        }
    }

    // A tile starts at a multiple of 64, so a key's slot is its own low bits,
    // and the tile's in blocks of 128.  A thread brings D / 4 values of key gt /
    // 4, and of V D / 64 values of the 16 tokens of granule `wave`.
    const int32_t *table = sq.table + (int64_t)b * sq.max_blocks;
    auto entry_at = [&](uint32_t t) { return table[min(t, k1 - 1) >> c.t_shift]; };    // as above
    auto block_of = [&](uint32_t t, int entry) {
        return t < k1 && entry >= 0 && entry < c.n_blocks ? entry : -1;
    };
    const int pk = gt >> 2, tv = 16 * wave + (lane & 15);   // the tokens whose z and s this thread brings
    uint32_t kr[NW], vr[NW], zk_raw, zv_raw;
    int k_entry, v_entry;
    bool k_ok, v_held, v_seen;              // whether the key's block, granule `wave`'s hold tokens; token tv is seen
    auto load_ids = [&](uint32_t tile) {
        k_entry = entry_at(tile + pk);
        v_entry = entry_at(tile + 16 * wave);
    };
    // what lies behind k1 is read from block 0
    auto load_tile = [&](uint32_t tile) {
        const int in = (int)tile & (c.T - 1);
        const int kid = block_of(tile + pk, k_entry), vid = block_of(tile + 16 * wave, v_entry);
        k_ok = kid >= 0;
        v_held = vid >= 0;
        v_seen = tile + tv < k1;
        const int64_t kt = (((int64_t)max(kid, 0) * c.KVH + h) << c.t_shift) + ((in + pk) & (c.T - 1));
        const int64_t vt = (((int64_t)max(vid, 0) * c.KVH + h) << c.t_shift) + ((in + 16 * wave) & (c.T - 1));
        const uint8_t *kp = c.K + kt * (D / 2) + D / 8 * (gt & 3), *vp = c.V + vt * (D / 2) + D / 8 * lane;
        if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(kp), y = *reinterpret_cast<const uint4 *>(vp);
            kr[0] = x.x; kr[1] = x.y; kr[NW - 2] = x.z; kr[NW - 1] = x.w;
            vr[0] = y.x; vr[1] = y.y; vr[NW - 2] = y.z; vr[NW - 1] = y.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(kp), y = *reinterpret_cast<const uint2 *>(vp);
            kr[0] = x.x; kr[1] = x.y;
            vr[0] = y.x; vr[1] = y.y;
        }
        zk_raw = c.zk[kt];
        zv_raw = c.zv[vt + (lane & 15)];
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
    constexpr int VD = D / 64;                              // values of V per thread
    const int k_put = k_at(pk, NW * (gt & 3)), v_put = v_at(VD * lane, 2 * wave);
    auto to_lds = [&](int buf) {
        const int ka = k_put + buf * kBuf, va = v_put + buf * kBuf;
        const uint32_t zk = k_ok ? sound(zk_raw) : 0u, zv = v_held && v_seen ? sound(zv_raw) : 0u;
        if (lane == 0) lds.held[buf][wave] = v_held;
        uint32_t sp[8], zp[8];
        // token t of 8 is half t / 4 of pair t % 4
        uint16_t *put = reinterpret_cast<uint16_t *>(lds.pairs[wave]) +
                        2 * (4 * ((lane >> 3) & 1) + (lane & 3)) + ((lane >> 2) & 1);
        if (lane < 16) {
            put[0] = (uint16_t)(zv >> 16);
            put[16] = (uint16_t)zv;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");           // one wave's LDS accesses are in order
        const uint4 *get = reinterpret_cast<const uint4 *>(lds.pairs[wave]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 w = get[i];
            uint32_t *to = i < 2 ? sp + 4 * i : zp + 4 * (i - 2);
            to[0] = w.x; to[1] = w.y; to[2] = w.z; to[3] = w.w;
        }
        const uint32_t ks = perm(zk, zk, 0x03020302u), kz = perm(zk, zk, 0x01000100u);
        const uint32_t ks4[4] = {ks, ks, ks, ks}, kz4[4] = {kz, kz, kz, kz};
#pragma unroll
        for (int j = 0; j < NW; ++j) *reinterpret_cast<half8 *>(lds_k + (ka ^ 16 * j)) = values8(kr[j], ks4, kz4);
#pragma unroll
        for (int j = 0; j < NW; ++j)
            *reinterpret_cast<half8 *>(lds_v + (va ^ 16 * (j & 1)) + (j >> 1) * 128) =
                values8(vr[j], sp + 4 * (j & 1), zp + 4 * (j & 1));
    };

    Reference ref;
    float l = 0.0f;
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
        // also where the wave's rows do not see the tile: one block to schedule
        float16v s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
        for (int st = 0; st < NQ; ++st) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const half8 k = *reinterpret_cast<const half8 *>(lds_k + (ka ^ 32 * st) + t * 64 * D);
                s[t] = mfma_32x32x16(k, qh[st], s[t]);
            }
        }
        to_lds(buf ^ 1);
        load_tile(tile + 2 * kTile);
        load_ids(tile + 3 * kTile);
        if (here) {
            const uint4 held = *reinterpret_cast<const uint4 *>(lds.held[buf]);
            const bool whole = __builtin_amdgcn_readfirstlane((held.x & held.y & held.z & held.w) != 0 &&
                                                              tile + kTile <= sees_lo);
            // of the tile's keys this lane's, 16 g + 8 half + e, are seen below lim = 16 g + e
            const int lim = (tile < sees ? (int)min(sees - tile, (uint32_t)kTile) : 0) - 8 * half;
            if (!whole) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int lim_g = (g == 0 ? held.x : g == 1 ? held.y : g == 2 ? held.z : held.w) ? lim : 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s[g >> 1][8 * (g & 1) + e] = 16 * g + e < lim_g ? s[g >> 1][8 * (g & 1) + e] : -INFINITY;
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, s[t][e]);
            float cs = c_row;                              // positive: q has the scale's sign
            top *= cs;
            if (__builtin_expect(__ballot(top > ref.above) != 0, 0)) {
                const float fix = ref.follow(half_max(top), 1.0f);
                l *= fix;
#pragma unroll
                for (int i = 0; i < NO; ++i) o[i] *= fix;
            }
            float base = ref.r1;
            if (__ballot(ref.far) != 0) {
                // r1 is exact for rows far from zero, and so is r1 with r2 = 0 for the others
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[t][e] = s[t][e] * cs - ref.r1;
                cs = 1.0f;
                base = ref.r2;
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {                  // 16 keys
                uint32_t w[4];
                float p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = exp2_fast(__builtin_fmaf(s[g >> 1][8 * (g & 1) + e], cs, -base));
                    l += p[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = f16_pair(p[e], p[e + 4]);
                const half8 ph = __builtin_bit_cast(half8, make_uint4(w[0], w[1], w[2], w[3]));
#pragma unroll
                for (int i = 0; i < NO; ++i) {
                    const half8 v = *reinterpret_cast<const half8 *>(lds_v + (va ^ 32 * g) + i * 32 * 128);
                    o[i] = mfma_32x32x16(v, ph, o[i]);
                }
            }
        }
        __syncthreads();
    }

    if (rw + low >= all_rows) return;
    l = l + __shfl_xor(l, 32);
    // from 2^(r1 + r2) to 2^r1
    float f0 = exp2_fast(ref.r2);
    l *= f0;
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
            if (direct) store4<true>(a.out, row * D + d, make_float4(y[0], y[1], y[2], y[3]));
            else store4<false>(dst, d, make_float4(y[0], y[1], y[2], y[3]));
        }
    if (!direct && half == 0) {
        float *ml = a.part + (int64_t)a.S * all * D + ((int64_t)split * all + row) * 2;
        ml[0] = ref.m == -INFINITY ? -INFINITY : ref.r1;
        ml[1] = l;
    }
}

template <bool BF16, int D>
__global__ __launch_bounds__(kThreads, 2) void kv4_few_kernel(Args a) {
    __shared__ FewLds<D> lds;
    few_rows<BF16, D>(a, blockIdx.x, lds);
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void kv4_many_kernel(Args a) {
    __shared__ ManyLds<D> lds;
    many_rows<D>(a, blockIdx.x, blockIdx.z, lds);
}
// Both in one launch: many rows wait for instructions, few rows for memory, so
// are to share the CUs.  The workgroups for few rows stand behind the first kCUs
// of the others.
template <int D>
__global__ __launch_bounds__(kThreads, 2) void kv4_mixed_kernel(Args a) {
    __shared__ union {
        FewLds<D> few;
        ManyLds<D> many;
    } lds;
    const int64_t all = a.many_groups * a.S, first = min(all, (int64_t)kCUs);
    const int64_t few = gridDim.x - all, i = blockIdx.x;
    if (i >= first && i < first + few) {
        few_rows<true, D>(a, (uint32_t)(i - first), lds.few);
    } else {
        const int64_t at = i < first ? i : i - few;
        const int split = (int)(at / a.many_groups);
        many_rows<D>(a, at - split * a.many_groups, split, lds.many);
    }
}

// By type.  bf16 rows, few and many, in us, tokens on keys of each sequence; 5 heads of 4
// with D = 128, and 8 heads of 2 with D = 64:
//   work  7680  4 x 256 on 1000      37.6  39.4     6144  22.7  34.5
//        11250  1000 on 1777         35.3  45.3     9000  21.7  35.7
//        15360  64 x 48 on 500       60.5  52.5    12288  34.6  32.2
//        15360  16 x 128 on 1000     67.0  54.4
//        17280  8 x 96 on 4000       69.6  89.0    13824  43.7  58.8
//        20320  128 on 32000         85.6   104    16256  55.0  48.0
//        21760  4 x 128 on 8000      95.3  86.1    17408  54.0  60.4
//        22500  1500 on 2500         62.7  70.1
//        25600  2048 on 2048         56.0  66.4
//        30720  64 x 96 on 500        112  72.4    24576  58.0  43.0
//        46080  2048 on 4096          124   124    36864  71.6  82.8
//        46080  64 x 32 on 4000       203   174    36864  99.7   153
//        92160  64 x 64 on 4000       344   296    73728   192   211
// No one bound suits all: many short sequences want the 128-row form from 12000 on, lone
// prompts and small heads on long keys not at 40000.  A workgroup of many rows for half
// the CUs only: 1000 rows on 1777 keys 57.8 us, for two a CU 46.7.  One sequence of more
// than 32 units for 256 pieces: 128 rows on 32000 keys 133 us, for 512 84.
constexpr Rules kRules[2] = {{1e30, kCUs, 32, 8}, {21000, 2 * kCUs, 32, 8}};

template <bool BF16, int D>
Kernels<Kv4Cache> kernels() {
    if constexpr (BF16) return {kv4_few_kernel<BF16, D>, kv4_many_kernel<D>, kv4_mixed_kernel<D>};
    else return {kv4_few_kernel<BF16, D>, nullptr, nullptr};
}

}  // namespace

size_t kv4_attention_ws_floats(int64_t n_tok, int64_t QH, int64_t B, int64_t max_blocks,
                               int64_t KVH, int64_t T, int64_t D) {
    size_t most = 0;                        // of the two types
    for (const Rules &r : kRules) {
        const Plan p = plan_for(n_tok, QH, B, max_blocks, KVH, T, D, r);
        const size_t need = (size_t)(p.part + p.cut);
        most = need > most ? need : most;
    }
    return most;
}

hipError_t launch_kv4_attention(const void *q, int dtype, int QH, const Kv8Seqs &seqs,
                                const bl_kv4 &cache, float scale, void *out, float *ws,
                                hipStream_t s) {
    const Plan p = plan_for(seqs.n_tok, QH, seqs.B, seqs.max_blocks, cache.KVH, cache.T, cache.D,
                            kRules[dtype]);
    const Args a = kv_args(p, q, QH, seqs, kv4_device(cache), scale, out, ws);
    if (cache.D == 64)
        return dtype ? attend<true, 64>(a, p, kernels<true, 64>(), s) : attend<false, 64>(a, p, kernels<false, 64>(), s);
    return dtype ? attend<true, 128>(a, p, kernels<true, 128>(), s) : attend<false, 128>(a, p, kernels<false, 128>(), s);
}

}  // namespace bl
