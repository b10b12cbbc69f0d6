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
// A code as fp16: the nibble put below 0x64 (0x54 where it stands four bits
// higher) reads as 1024 + u (64 + u); one packed add leaves u.  Eight codes of a
// dword come out as the pairs (0, 4) (1, 5) (2, 6) (3, 7): a product's order of
// terms is free, so q and the weights are put into that order instead.
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

// Eight codes -> fp16, pairs (0, 4) (1, 5) (2, 6) (3, 7).
__device__ __forceinline__ half8 codes8(uint32_t w) {
    const half2 b0 = {(_Float16)-1024.0f, (_Float16)-1024.0f}, b1 = {(_Float16)-64.0f, (_Float16)-64.0f};
    const uint32_t v = w >> 8;
    uint4 o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, (w & 0x000F000Fu) | 0x64006400u) + b0);
    o.y = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, (w & 0x00F000F0u) | 0x54005400u) + b1);
    o.z = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, (v & 0x000F000Fu) | 0x64006400u) + b0);
    o.w = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, (v & 0x00F000F0u) | 0x54005400u) + b1);
    return __builtin_bit_cast(half8, o);
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
    template <bool BF16>
    __device__ __forceinline__ float follow(float top, float u_new) {
        const bool none = m == -INFINITY;
        m = fmaxf(m, top);
        u = u_new;
        above = raise_above<BF16>(m);
        const float base = m == -INFINITY ? 0.0f : m, shift = log2_of(u) - kUnitBits;
        far = fabsf(base) >= kFarScore<BF16>;
        const float n1 = far ? base : base + shift, n2 = far ? shift : 0.0f;
        const float fix = none ? 0.0f : exp2_fast((r1 - n1) + (r2 - n2));
        r1 = n1;
        r2 = n2;
        return fix;
    }
};

// Few rows: one workgroup to a piece; its waves take 64-key tiles in turn, each
// with sums of its own, joined in LDS.  Operands go from memory to registers:
// a cached byte has one reader.  The next tile's K is under way from the
// moment this one's has been used, and so is V.
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
        q_sum = quad_sum(q_sum) * a.scale2;
        const float f = a.scale2 < 0.0f ? -to_f16_range(top) : to_f16_range(top);
        c_row = a.scale2 / f;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const float x[8] = {v[j][0].x * f, v[j][0].y * f, v[j][0].z * f, v[j][0].w * f,
                                v[j][1].x * f, v[j][1].y * f, v[j][1].z * f, v[j][1].w * f};
            uint32_t w[4], z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = f16_pair(x[e], x[e + 4]);
                z[e] = f16_rest(x[e], x[e + 4], w[e]);
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
            float x[16];                    // scores of the quad's tokens, in powers of two
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                float4v s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const half8 k = codes8(kb[tt][j]);
#pragma unroll
                    for (int e = 0; e < NS; ++e) s = mfma_16x16x32(k, qh[e][j], s);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t zs = zk[4 * tt + i];
                    x[4 * tt + i] = __builtin_fmaf(s[i] * c_row, (float)zs_s(zs),
                                                   __builtin_fmaf(q_sum, (float)zs_z(zs), 0.0f));
                }
            }
            const uint32_t next = tile + kStep;
            const bool more = next < k1;
            if (more) {
                id_next = block_of(next, entry);
                load_k(next, id_next);
            }

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
            top = quad_max(top);
            const float u_new = fmaxf(ref.u, step_above(quad_max((float)zs_s(zs_top))));
            if (__builtin_expect(__ballot(top > ref.above || u_new != ref.u) != 0, 0)) {
                const float fix = ref.follow<BF16>(top, u_new);
                l *= fix;
                o_z *= fix;
#pragma unroll
                for (int i = 0; i < NO; ++i) o[i] *= fix;
            }
            const float base = ref.far ? ref.r2 : ref.r1;
            if (__ballot(ref.far) != 0) {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] -= ref.far ? ref.r1 : 0.0f;
            }
            half8 ph[NS][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t hi[4], lo[4];
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t zs = zv[8 * k + e];
                    const float p = exp2_fast(x[8 * k + e] - base);
                    l += p;
                    o_z = __builtin_fmaf(p, (float)zs_z(zs), o_z);
                    y[e] = __builtin_fmaf(p, (float)zs_s(zs), 0.0f);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hi[e] = f16_pair(y[e], y[e + 4]);
                    if (!BF16) lo[e] = f16_rest(y[e], y[e + 4], hi[e]);
                }
                ph[0][k] = __builtin_bit_cast(half8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                if (!BF16) ph[NS - 1][k] = __builtin_bit_cast(half8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
#pragma unroll
            for (int i = 0; i < NO / 2; ++i) {
                const half8 v00 = codes8(vb[i].x), v01 = codes8(vb[i].y);
                const half8 v10 = codes8(vb[i].z), v11 = codes8(vb[i].w);
#pragma unroll
                for (int e = 0; e < NS; ++e) {
                    o[2 * i] = mfma_16x16x32(v00, ph[e][0], o[2 * i]);
                    o[2 * i + 1] = mfma_16x16x32(v10, ph[e][0], o[2 * i + 1]);
                    o[2 * i] = mfma_16x16x32(v01, ph[e][1], o[2 * i]);
                    o[2 * i + 1] = mfma_16x16x32(v11, ph[e][1], o[2 * i + 1]);
                }
            }
            if (more) {
                id = id_next;
                entry = entry_at(next + kStep);            // before V: loads come back in order
                load_v(next, id);
            }
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
            join[wave][low][32 * (i / 2) + 2 * (4 * quad + e) + (i & 1)] = (o[i][e] + o_z) * f_r2;
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

template <bool BF16, int D>
__global__ __launch_bounds__(kThreads, 2) void kv4_few_kernel(Args a) {
    __shared__ FewLds<D> lds;
    few_rows<BF16, D>(a, blockIdx.x, lds);
}

template <bool BF16, int D>
Kernels<Kv4Cache> kernels() {
    return {kv4_few_kernel<BF16, D>, nullptr, nullptr};
}

}  // namespace

size_t kv4_attention_ws_floats(int64_t n_tok, int64_t QH, int64_t B, int64_t max_blocks,
                               int64_t KVH, int64_t T, int64_t D) {
    const Plan p = plan_for(n_tok, QH, B, max_blocks, KVH, T, D, false);
    return (size_t)(p.part + p.cut);
}

hipError_t launch_kv4_attention(const void *q, int dtype, int QH, const Kv8Seqs &seqs,
                                const bl_kv4 &cache, float scale, void *out, float *ws,
                                hipStream_t s) {
    const Plan p = plan_for(seqs.n_tok, QH, seqs.B, seqs.max_blocks, cache.KVH, cache.T, cache.D, false);
    const Args a = kv_args(p, q, QH, seqs, kv4_device(cache), scale, out, ws);
    if (cache.D == 64)
        return dtype ? attend<true, 64>(a, p, kernels<true, 64>(), s) : attend<false, 64>(a, p, kernels<false, 64>(), s);
    return dtype ? attend<true, 128>(a, p, kernels<true, 128>(), s) : attend<false, 128>(a, p, kernels<false, 128>(), s);
}

}  // namespace bl
