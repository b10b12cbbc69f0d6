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
#include "kv_attention.h"

namespace bl {
namespace {

using Args = KvArgs<Kv8Cache>;

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

// A single sequence is always cut where that may save steps: one token on 4000 keys in a
// captured call of 128 rows takes 9.3 us, uncut 26.5 (128 tokens 32.2, without a join 29.8).
constexpr Rules kRules = {kManyWork, kCUs, INT32_MAX, 0};

template <bool BF16, int D>
Kernels<Kv8Cache> kernels() {
    return {kv8_few_kernel<BF16, D>, kv8_many_kernel<BF16, D>, kv8_mixed_kernel<BF16, D>};
}

}  // namespace

size_t kv8_attention_ws_floats(int64_t n_tok, int64_t QH, int64_t B, int64_t max_blocks,
                               int64_t KVH, int64_t T, int64_t D) {
    const Plan p = plan_for(n_tok, QH, B, max_blocks, KVH, T, D, kRules);
    return (size_t)(p.part + p.cut);
}

hipError_t launch_kv8_attention(const void *q, int dtype, int QH, const Kv8Seqs &seqs,
                                const bl_kv8 &cache, float scale, void *out, float *ws,
                                hipStream_t s) {
    const Plan p = plan_for(seqs.n_tok, QH, seqs.B, seqs.max_blocks, cache.KVH, cache.T, cache.D,
                            kRules);
    const Args a = kv_args(p, q, QH, seqs, kv8_device(cache), scale, out, ws);
    if (cache.D == 64)
        return dtype ? attend<true, 64>(a, p, kernels<true, 64>(), s) : attend<false, 64>(a, p, kernels<false, 64>(), s);
    return dtype ? attend<true, 128>(a, p, kernels<true, 128>(), s) : attend<false, 128>(a, p, kernels<false, 128>(), s);
}

}  // namespace bl
