// kv_attention.cu -- attention of new tokens over the paged 8-bit K/V cache.
//
// For a new token at position p of its sequence and query head h of the key head's group:
//   s_t = scale * d_K(t) * (q . c_K(t)),  t <= p (causal) or t < length
//   y   = sum_t exp(s_t) d_V(t) c_V(t) / sum_t exp(s_t),   lse = log sum_t exp(s_t)
// in one pass with a running maximum and sum, all in fp32.  A row that sees nothing gives zeros and
// lse -inf.
//
// One warp a row: lanes take tokens for the scores and features for the output.
#include "kv_common.cuh"

namespace bitnet {
namespace {

template <int D>
__global__ void __launch_bounds__(128)
    kv_attention_rows_kernel(KvArgs a, AttentionArgs at) {
    constexpr int F = D / 32;  // features a lane
    __shared__ float qs[4][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 4 + warp;
    if (row >= (int64_t)a.tokens * at.q_heads) return;
    const int token = (int)(row / at.q_heads), qh = (int)(row - (int64_t)token * at.q_heads);
    const int s = find_sequence(token, a.batch, [&](int i) { return (int64_t)__ldg(a.q_start + i); });
    const KvSequence q = kv_sequence(a, s);
    if (!q.valid || q.count > at.max_new) {
        if (lane == 0) record_status(a.status, BITNET_ERR_INVALID);
        return;
    }
    const int i = token - q.first;
    if (i < 0 || i >= q.count) return;  // a row of no sequence
    const int seen = at.causal ? q.length - q.count + i + 1 : q.length;
    const int head = qh / (at.q_heads / a.kv_heads);
    const __nv_bfloat16 *Q = reinterpret_cast<const __nv_bfloat16 *>(at.Q) + token * at.ldq + qh * D;
    for (int f = lane; f < D; f += 32) qs[warp][f] = __bfloat162float(Q[f]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[F] = {};
    for (int t0 = 0; t0 < seen; t0 += 32) {
        const int t = t0 + lane;
        float sc = -INFINITY, dv = 0.f;
        const int8_t *v = nullptr;
        if (t < seen) {
            const int page = kv_page(a, s, t);
            if (page >= 0) {
                const int64_t c = kv_code_at(a, page, head, t), d = kv_scale_at(a, page, head, t);
                float dot = 0.f;
                for (int f = 0; f < D; ++f) dot += qs[warp][f] * (float)a.k_codes[c + f];
                sc = dot * a.k_scales[d] * at.scale;
                dv = a.v_scales[d];
                v = a.v_codes + c;
            }
        }
        float mt = sc;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, x));
        const float mn = fmaxf(m, mt);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float p = v ? __expf(sc - base) : 0.f, keep = __expf(m - base);
        float sum = p;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        l = l * keep + sum;
        m = mn;
#pragma unroll
        for (int f = 0; f < F; ++f) o[f] *= keep;
        for (int j = 0; j < 32; ++j) {
            const float w = __shfl_sync(0xFFFFFFFFu, v ? p * dv : 0.f, j);
            const int8_t *vj = reinterpret_cast<const int8_t *>(
                __shfl_sync(0xFFFFFFFFu, (unsigned long long)v, j));
            if (vj)
#pragma unroll
                for (int f = 0; f < F; ++f) o[f] += w * (float)vj[f * 32 + lane];
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16 *Y = reinterpret_cast<__nv_bfloat16 *>(at.Y) + token * at.ldy + qh * D;
#pragma unroll
    for (int f = 0; f < F; ++f) Y[f * 32 + lane] = __float2bfloat16(o[f] * inv);
    if (at.lse && lane == 0)
        at.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t kv_attention_workspace(const KvArgs &a, const AttentionArgs &at) {
    (void)a;
    (void)at;
    return 0;
}

cudaError_t launch_kv_attention(const KvArgs &a, const AttentionArgs &at, void *ws,
                                cudaStream_t stream, int *launches) {
    (void)ws;
    const int64_t rows = (int64_t)a.tokens * at.q_heads, blocks = (rows + 3) / 4;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    *launches = 1;
    auto kern = a.head_dim == 64 ? kv_attention_rows_kernel<64> : kv_attention_rows_kernel<128>;
    kern<<<(unsigned)blocks, 128, 0, stream>>>(a, at);
    return cudaGetLastError();
}

}  // namespace bitnet
