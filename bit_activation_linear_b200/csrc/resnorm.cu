// resnorm.cu -- the residual stream's step between two sub-layers: residual addition, RMS
// normalisation and per-token activation codes in one pass.
//
// BitNet b1.58 2B4T article, section 一.3 (subln / RMS normalisation in front of the quantised
// projections).  Per token row, with x the sub-layer's output and r the residual stream (bf16):
//   h = bf16_rn(x + r)                                  (the new residual stream, stored)
//   y = (h * rinv) * g,  rinv = 1 / sqrt(sum h^2 / K + eps)   (each an IEEE fp32 operation)
//   codes of y: absmax INT8 or absmean INT4, as act_quant_plain_kernel.
// The norm reads the ROUNDED h: it is what the stream holds and what every later reader sees, so
// one call gives what the addition followed by bitnet_act_quant_norm gives.  One thing differs: a NaN
// or an infinity of a row reaches its scale (and its codes are 0), so that products with the row are
// NaN and not small plausible numbers.
//
// Bound by HBM: 6 bytes and the code an element, read once.  A row stays in the registers of its
// threads between the addition and the codes (4 chunks of 8 values each, so K / 32 threads a row).
// Measured on B200: 16383 x 4096 in 72 .. 76 us (5.9 .. 6.5 TB/s), 4096 x 2048 in 13 .. 14 us, one row in
// the 3.4 us of a launch.  INT4 takes 83 us for the first: its mean is summed in double, as every
// absmean of this library, and the conversions (two a value) bound it.  Rows above K = 32768 need more
// threads than a block has and are read back: 4.5 TB/s at 33024 against 4.9 TB/s at 32768.
#include "common.cuh"
#include "kernels.h"

namespace bitnet {
namespace {

constexpr float kSqrt7 = 2.6457513110645906f;  // code of the mean magnitude (INT4)

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    // fp32 sums, each rounded once to bf16
    const float lo = __fadd_rn(__uint_as_float(a << 16), __uint_as_float(b << 16));
    const float hi = __fadd_rn(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u));
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // fmaxf would drop a NaN
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The eight normalised values of a chunk of h.
__device__ __forceinline__ void normalise8(const uint4 &h4, const uint4 &g4, float rinv,
                                           float2 (&y)[4]) {
    const uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w}, g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = mul2_rn(mul2_rn(make_float2(__uint_as_float(h[i] << 16),
                                           __uint_as_float(h[i] & 0xFFFF0000u)),
                               make_float2(rinv, rinv)),
                       make_float2(__uint_as_float(g[i] << 16),
                                   __uint_as_float(g[i] & 0xFFFF0000u)));
}

// blockDim.x = rows * tpr: each row of K is taken by tpr threads (a multiple of 32), CH chunks of
// 8 values a thread, kept in registers as bf16 from the one read to the codes.  CH = 0: rows too
// long for that; h is read back from global memory (each thread reads what it wrote).
template <int BITS, int CH>
__global__ void __launch_bounds__(1024)
    residual_norm_quant_kernel(const uint4 *X, const uint4 *R, int64_t M, int K, int tpr,
                               const uint4 *__restrict__ gain, float eps, uint4 *H,
                               uint8_t *__restrict__ codes, float *__restrict__ scales,
                               int32_t *__restrict__ rowsum) {
    __shared__ float red_ss[32];
    __shared__ double red_abs[32];
    __shared__ int red_sum[32];
    pdl_launch_dependents();
    const int local = threadIdx.x / tpr, tid = threadIdx.x - local * tpr;
    const int lane = threadIdx.x & 31, warps = tpr / 32, warp0 = local * warps;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + local;
    const bool live = row < M;  // idle rows of the last block still meet the barriers
    const int nchunk = live ? K / 8 : 0;
    const int64_t base = row * (K / 8);
    const uint4 unit = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);

    constexpr int KEEP = CH > 0 ? CH : 1;
    uint4 h[KEEP];
    float ss = 0.f;
    auto add = [&](const uint4 &x, const uint4 &r, int c) {
        uint4 v;
        v.x = add_bf16x2(x.x, r.x);
        v.y = add_bf16x2(x.y, r.y);
        v.z = add_bf16x2(x.z, r.z);
        v.w = add_bf16x2(x.w, r.w);
        H[base + c] = v;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
            ss = __fmaf_rn(a, a, ss);
            ss = __fmaf_rn(b, b, ss);
        }
        return v;
    };
    if constexpr (CH > 0) {
        uint4 x[KEEP], r[KEEP];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = tid + i * tpr;
            if (c < nchunk) {
                x[i] = X[base + c];
                r[i] = R[base + c];
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = tid + i * tpr;
            if (c < nchunk) h[i] = add(x[i], r[i], c);
        }
    } else {
        for (int c = tid; c < nchunk; c += tpr) add(X[base + c], R[base + c], c);
    }
    // visits the row's normalised values
    auto each = [&](float rinv, auto &&f) {
        if constexpr (CH > 0) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = tid + i * tpr;
                if (c < nchunk) {
                    float2 y[4];
                    normalise8(h[i], gain ? __ldg(gain + c) : unit, rinv, y);
                    f(c, y);
                }
            }
        } else {
            for (int c = tid; c < nchunk; c += tpr) {
                float2 y[4];
                normalise8(H[base + c], gain ? __ldg(gain + c) : unit, rinv, y);
                f(c, y);
            }
        }
    };

#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (warps > 1) {
        if (lane == 0) red_ss[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = lane < warps ? red_ss[warp0 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    }
    const float rinv = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)K), eps)));

    float g;
    constexpr float Q = BITS == 4 ? kSqrt7 : 127.f;
    if constexpr (BITS == 4) {
        double sa = 0.0;  // in double, as every absmean of this library
        each(rinv, [&](int, float2 (&y)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sa += fabs((double)y[i].x) + fabs((double)y[i].y);
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sa += __shfl_xor_sync(0xFFFFFFFFu, sa, o);
        if (warps > 1) {
            if (lane == 0) red_abs[threadIdx.x >> 5] = sa;
            __syncthreads();
            sa = lane < warps ? red_abs[warp0 + lane] : 0.0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sa += __shfl_xor_sync(0xFFFFFFFFu, sa, o);
        }
        const double mean = sa / (double)K;
        g = (float)(mean < 1e-5 ? 1e-5 : mean);  // keeps NaN
    } else {
        float most = 0.f;
        each(rinv, [&](int, float2 (&y)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) most = max_nan(most, max_nan(fabsf(y[i].x), fabsf(y[i].y)));
        });
        // non-negative floats order like their bit patterns, NaN above everything
        uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most) & 0x7FFFFFFFu);
        if (warps > 1) {
            uint32_t *red = reinterpret_cast<uint32_t *>(red_abs);
            if (lane == 0) red[threadIdx.x >> 5] = m;
            __syncthreads();
            m = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? red[warp0 + lane] : 0u);
        }
        const float mx = __uint_as_float(m);
        g = mx < 1e-5f ? 1e-5f : mx;
    }
    const float s = __fdiv_rn(Q, g);
    const uint32_t keep = g <= 3.4028235e38f ? 0xFFFFFFFFu : 0u;  // codes of 0 beside a NaN or inf
    const float2 magic2 = make_float2(12582912.f, 12582912.f);  // 1.5 * 2^23: round to integer
    int sum = 0;
    each(rinv, [&](int c, float2 (&y)[4]) {
        uint32_t f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the products that decide codes are never contracted with the rounding add
            float2 t = make_float2(__fmul_rn(y[i].x, s), __fmul_rn(y[i].y, s));
            if constexpr (BITS == 4)
                t = make_float2(fminf(fmaxf(t.x, -8.f), 7.f), fminf(fmaxf(t.y, -8.f), 7.f));
            const float2 u = __fadd2_rn(t, magic2);
            f[2 * i] = __float_as_uint(u.x);
            f[2 * i + 1] = __float_as_uint(u.y);
        }
        const uint32_t A = gather_low_bytes(f[0], f[1], f[2], f[3]) & keep;
        const uint32_t B = gather_low_bytes(f[4], f[5], f[6], f[7]) & keep;
        sum = __dp4a((int)A, 0x01010101, sum);
        sum = __dp4a((int)B, 0x01010101, sum);
        if constexpr (BITS == 8)
            *reinterpret_cast<uint2 *>(codes + row * K + 8 * c) = make_uint2(A, B);
        else
            *reinterpret_cast<uint32_t *>(codes + row * (K / 2) + 4 * c) =
                (A & 0x0F0F0F0Fu) | ((B << 4) & 0xF0F0F0F0u);
    });
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    if (warps > 1) {
        if (lane == 0) red_sum[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = __reduce_add_sync(0xFFFFFFFFu, lane < warps ? red_sum[warp0 + lane] : 0);
    }
    if (live && tid == 0) {
        scales[row] = __fdiv_rn(g, Q);
        rowsum[row] = sum;
    }
}

}  // namespace

cudaError_t launch_residual_norm_quant(const void *X, const void *R, int64_t M, int64_t K,
                                       int act_bits, const NormArgs &nrm, void *H, void *codes,
                                       float *scales, int32_t *rowsum, cudaStream_t stream) {
    const int nchunk = (int)(K / 8);
    auto go = [&](auto kern, int tpr) {
        const int rows = tpr >= 128 ? 1 : 128 / tpr;
        kern<<<(unsigned)((M + rows - 1) / rows), rows * tpr, 0, stream>>>(
            reinterpret_cast<const uint4 *>(X), reinterpret_cast<const uint4 *>(R), M, (int)K, tpr,
            reinterpret_cast<const uint4 *>(nrm.gain), nrm.eps, reinterpret_cast<uint4 *>(H),
            reinterpret_cast<uint8_t *>(codes), scales, rowsum);
        return cudaGetLastError();
    };
    auto threads = [&](int ch) { return ((nchunk + ch - 1) / ch + 31) / 32 * 32; };
    if (act_bits == 4) {
        if (nchunk <= 4 * 1024) return go(residual_norm_quant_kernel<4, 4>, threads(4));
        return go(residual_norm_quant_kernel<4, 0>, 1024);
    }
    if (nchunk <= 4 * 1024) return go(residual_norm_quant_kernel<8, 4>, threads(4));
    return go(residual_norm_quant_kernel<8, 0>, 1024);
}

}  // namespace bitnet
