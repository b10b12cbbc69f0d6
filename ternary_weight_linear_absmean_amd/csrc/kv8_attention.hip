// kv8_attention.hip -- causal attention over the 8-bit key/value cache.
//
// out = sum_j p_j v_j / sum_j p_j, p_j = exp(s_j - max s), s_j = scale q.k_j,
// in one pass over the keys with a running maximum.  One wave per (row, query
// head), a lane holding D / 64 of the values.
#include "kv8_common.h"

namespace bl {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__global__ __launch_bounds__(kThreads) void kv8_attention_kernel(const void *__restrict__ q, int QH,
                                                                 Kv8Seqs seqs, Kv8Cache c,
                                                                 float scale, void *out) {
    const int lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (i >= (int64_t)seqs.n_tok * QH) return;
    const int t = (int)(i / QH), hq = (int)(i % QH), h = hq / (QH / c.KVH);
    const int b = find_seq(seqs.B, t, [&](int x) { return (int64_t)q_at(seqs, x); });
    const int q0 = q_at(seqs, b), q1 = q_at(seqs, b + 1);
    if (t < q0 || t >= q1) return;
    const int64_t pos = (int64_t)seqs.lengths[b] - (q1 - t);
    const int per = c.D / 64;
    float x[2], o[2] = {0.0f, 0.0f}, m = -INFINITY, l = 0.0f;
    for (int e = 0; e < per; ++e) {
        const int64_t at = i * c.D + e * 64 + lane;
        x[e] = BF16 ? bf16_lo(static_cast<const uint16_t *>(q)[at]) : static_cast<const float *>(q)[at];
    }
    const int64_t end = min(pos + 1, (int64_t)seqs.max_blocks << c.t_shift);
    for (int64_t j = 0; j < end; ++j) {
        const int id = seqs.table[(int64_t)b * seqs.max_blocks + (j >> c.t_shift)];
        if (id < 0 || id >= c.n_blocks) continue;
        const int64_t hb = (int64_t)id * c.KVH + h;
        const int slot = (int)j & (c.T - 1);
        float s = 0.0f;
        for (int e = 0; e < per; ++e)
            s += x[e] * (float)c.K[hb * c.T * c.D + slot * c.D + e * 64 + lane];
        for (int w = 1; w < 64; w <<= 1) s += __shfl_xor(s, w);
        s = s * c.sk[hb] * scale;
        const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
        for (int e = 0; e < per; ++e)
            o[e] = o[e] * f +
                   p * ((float)c.V[hb * c.T * c.D + (e * 64 + lane) * c.T + slot] * c.sv[hb]);
    }
    for (int e = 0; e < per; ++e) {
        const int64_t at = i * c.D + e * 64 + lane;
        const float y = l > 0.0f ? o[e] / l : 0.0f;
        if (BF16) {
            const uint32_t w = __float_as_uint(y);
            static_cast<uint16_t *>(out)[at] = (uint16_t)((w + 0x7FFF + (w >> 16 & 1)) >> 16);
        } else {
            static_cast<float *>(out)[at] = y;
        }
    }
}

}  // namespace

size_t kv8_attention_ws_floats(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) {
    return 0;
}

hipError_t launch_kv8_attention(const void *q, int dtype, int QH, const Kv8Seqs &seqs,
                                const bl_kv8 &cache, float scale, void *out, float *ws,
                                hipStream_t s) {
    const Kv8Cache c = kv8_device(cache);
    const dim3 grid((unsigned)(((int64_t)seqs.n_tok * QH + 3) / 4)), block(kThreads);
    if (dtype)
        hipLaunchKernelGGL(kv8_attention_kernel<true>, grid, block, 0, s, q, QH, seqs, c, scale, out);
    else
        hipLaunchKernelGGL(kv8_attention_kernel<false>, grid, block, 0, s, q, QH, seqs, c, scale, out);
    return hipGetLastError();
}

}  // namespace bl
