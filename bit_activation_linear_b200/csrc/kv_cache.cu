// kv_cache.cu -- the paged 8-bit K/V cache: states quantised as they are written, and read back.
//
// BitNet v2 write-up, Tables 2 and 3: the attention's K and V states are kept in few bits.  Here
// they are kept in 8, with one fp32 step d for each block of `block` tokens (16 .. a page) of one
// head: x ~ c * d.  Writing new tokens into a block (absmax over the block, fp32):
//   mx    = max(max |x| over the block's new tokens and the head's features, 1e-5)
//   g_old = 127 * d_old, or 0 when the block's first token is among the new ones (a page that
//           came back from another sequence keeps nothing)
//   mx > g_old:  g = mx, d = g / 127, and the block's older codes become rint(c * (d_old * s));
//   else         g = g_old, d = d_old;
//   s = 127 / g, c = clip(rint(x * s), -127, 127).
// A block whose step grows rounds its older codes once more (by at most half the new step).
//
// A NaN or an infinity makes its block's step NaN or infinite (the maximum is taken on the bit
// patterns, which order NaN above everything) until the block is written anew: attention over it
// gives NaN instead of a plausible number.
#include "kv_common.cuh"

namespace bitnet {
namespace {

// Work items are (block of a sequence that gets new tokens, state K or V, head), one warp each.
// Sequence s owns the items from first(s) / block + 2 s on: that is non-decreasing, leaves room
// for the blocks that n tokens can touch (n / block + 2), and needs no prefix sum.
constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t max_bits(uint32_t m, const uint4 &v) {
    m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

// cvt.rni saturates and turns NaN into 0
__device__ __forceinline__ uint32_t code(float x, float s) {
    return (uint32_t)max(min(__float2int_rn(__fmul_rn(x, s)), 127), -127) & 0xFFu;
}

__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float s) {
    return code(__uint_as_float(a << 16), s) | code(__uint_as_float(a & 0xFFFF0000u), s) << 8 |
           code(__uint_as_float(b << 16), s) << 16 | code(__uint_as_float(b & 0xFFFF0000u), s) << 24;
}

__device__ __forceinline__ uint32_t recode4(uint32_t c, float r) {
    uint32_t d = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) d |= code((float)(int8_t)(c >> (8 * i)), r) << (8 * i);
    return d;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps)
    kv_append_kernel(KvArgs a, const uint8_t *__restrict__ K, int64_t ldk,
                     const uint8_t *__restrict__ V, int64_t ldv, int64_t items) {
    constexpr int LPT = D / 8;       // lanes a token: 16 bytes of bf16 each
    constexpr int TPW = 32 / LPT;    // tokens the warp reads at once
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= items) return;
    const int per_block = 2 * a.kv_heads;
    const int64_t w = item / per_block;
    const int which = (int)(item - w * per_block) / a.kv_heads;
    const int head = (int)(item - w * per_block) - which * a.kv_heads;
    auto begin = [&](int s) {
        return (int64_t)(__ldg(a.q_start + s) >> a.block_shift) + 2 * (int64_t)s;
    };
    const int s = find_sequence(w, a.batch, begin);
    const KvSequence q = kv_sequence(a, s);
    if (!q.valid || q.count > q.length) {  // nothing of such a sequence is written
        if (lane == 0) record_status(a.status, BITNET_ERR_INVALID);
        return;
    }
    const int block = 1 << a.block_shift, p0 = q.length - q.count;
    const int64_t j = w - begin(s);
    if (j < 0 || q.count == 0) return;
    const int64_t start = ((int64_t)(p0 >> a.block_shift) + j) << a.block_shift;
    if (start >= q.length) return;
    const int lo = max(p0, (int)start), hi = min((int64_t)q.length, start + block);
    const int page = kv_page(a, s, (int)start);
    if (page < 0) return;
    int8_t *out = (which ? a.v_codes : a.k_codes) + kv_code_at(a, page, head, (int)start);
    float *step = (which ? a.v_scales : a.k_scales) + kv_scale_at(a, page, head, (int)start);
    const int64_t ld = 2 * (which ? ldv : ldk);  // bytes a token row
    const uint8_t *in = (which ? V : K) + (int64_t)(q.first + lo - p0) * ld + 2 * head * D;
    const int sub = lane / LPT, off = lane % LPT, count = hi - lo;

    uint32_t m = 0;
    for (int t = sub; t < count; t += TPW)
        m = max_bits(m, __ldg(reinterpret_cast<const uint4 *>(in + t * ld) + off));
    m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
    float mx = __uint_as_float(m << 16);
    if (mx < 1e-5f) mx = 1e-5f;  // keeps NaN
    const float d_old = lo > start ? *step : 0.f;
    const float g_old = __fmul_rn(127.f, d_old);
    const bool grown = !(mx <= g_old) && !isnan(g_old);
    const float g = grown ? mx : g_old;
    const float s8 = __fdiv_rn(127.f, g);
    if (grown && lo > start) {  // the block's older codes, with the new step
        const float r = __fmul_rn(d_old, s8);
        uint4 *old = reinterpret_cast<uint4 *>(out);
        for (int i = lane; i < (lo - (int)start) * D / 16; i += 32) {
            uint4 c = old[i];
            c.x = recode4(c.x, r);
            c.y = recode4(c.y, r);
            c.z = recode4(c.z, r);
            c.w = recode4(c.w, r);
            old[i] = c;
        }
    }
    uint2 *dst = reinterpret_cast<uint2 *>(out + (lo - (int)start) * D);
    for (int t = sub; t < count; t += TPW) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(in + t * ld) + off);
        dst[t * LPT + off] = make_uint2(codes4(x.x, x.y, s8), codes4(x.z, x.w, s8));
    }
    __syncwarp();  // every lane has read the old step
    if (lane == 0 && grown) *step = __fdiv_rn(g, 127.f);
}

// Reads back a sequence's last tokens, 16 positions of one head a warp.  A block is at least 16
// tokens, so the 16 share a step.
constexpr int kReadShift = 4;

__device__ __forceinline__ uint32_t value2(uint32_t two, float d) {  // two codes -> two bf16
    const float lo = __fmul_rn((float)(int8_t)two, d);
    const float hi = __fmul_rn((float)(int8_t)(two >> 8), d);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps)
    kv_read_kernel(KvArgs a, uint8_t *__restrict__ K, int64_t ldk, uint8_t *__restrict__ V,
                   int64_t ldv, int64_t items) {
    constexpr int LPT = D / 8, TPW = 32 / LPT;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= items) return;
    const int per_block = 2 * a.kv_heads;
    const int64_t w = item / per_block;
    const int which = (int)(item - w * per_block) / a.kv_heads;
    const int head = (int)(item - w * per_block) - which * a.kv_heads;
    auto begin = [&](int s) { return (int64_t)(__ldg(a.q_start + s) >> kReadShift) + 2 * (int64_t)s; };
    const int s = find_sequence(w, a.batch, begin);
    const KvSequence q = kv_sequence(a, s);
    if (!q.valid || q.count > q.length) {
        if (lane == 0) record_status(a.status, BITNET_ERR_INVALID);
        return;
    }
    const int p0 = q.length - q.count;
    const int64_t j = w - begin(s);
    if (j < 0 || q.count == 0) return;
    const int64_t start = ((int64_t)(p0 >> kReadShift) + j) << kReadShift;
    if (start >= q.length) return;
    const int lo = max(p0, (int)start), hi = min((int64_t)q.length, start + (1 << kReadShift));
    const int page = kv_page(a, s, (int)start);
    if (page < 0) return;
    const uint2 *in = reinterpret_cast<const uint2 *>((which ? a.v_codes : a.k_codes) +
                                                      kv_code_at(a, page, head, lo));
    const float d = (which ? a.v_scales : a.k_scales)[kv_scale_at(a, page, head, (int)start)];
    const int64_t ld = 2 * (which ? ldv : ldk);
    uint8_t *out = (which ? V : K) + (int64_t)(q.first + lo - p0) * ld + 2 * head * D;
    const int sub = lane / LPT, off = lane % LPT;
#pragma unroll 4
    for (int t = sub; t < hi - lo; t += TPW) {
        const uint2 c = in[t * LPT + off];
        reinterpret_cast<uint4 *>(out + t * ld)[off] =
            make_uint4(value2(c.x, d), value2(c.x >> 16, d), value2(c.y, d), value2(c.y >> 16, d));
    }
}

}  // namespace

static int64_t kv_items(const KvArgs &a, int shift) {
    return (((int64_t)a.tokens >> shift) + 2 * (int64_t)a.batch) * 2 * a.kv_heads;
}

cudaError_t launch_kv_append(const KvArgs &a, const void *K, int64_t ldk, const void *V,
                             int64_t ldv, cudaStream_t stream) {
    const int64_t items = kv_items(a, a.block_shift);
    const int64_t blocks = (items + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    auto kern = a.head_dim == 64 ? kv_append_kernel<64> : kv_append_kernel<128>;
    kern<<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(a, static_cast<const uint8_t *>(K), ldk,
                                                       static_cast<const uint8_t *>(V), ldv, items);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvArgs &a, void *K, int64_t ldk, void *V, int64_t ldv,
                           cudaStream_t stream) {
    const int64_t items = kv_items(a, kReadShift);
    const int64_t blocks = (items + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    auto kern = a.head_dim == 64 ? kv_read_kernel<64> : kv_read_kernel<128>;
    kern<<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(a, static_cast<uint8_t *>(K), ldk,
                                                       static_cast<uint8_t *>(V), ldv, items);
    return cudaGetLastError();
}

}  // namespace bitnet
