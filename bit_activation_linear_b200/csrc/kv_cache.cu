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
// Both kernels move 3 bytes a state and are bound by HBM for many tokens (read back of 44 000 tokens
// of 8 heads: 49 us, 5.6 TB/s), by launch and dependent loads for few (one token for each of 64
// sequences: 3.7 us; 8700 tokens: 14 us).
#include "kv_common.cuh"

namespace bitnet {
namespace {

// A block takes a span of positions of one sequence (64 or a longer scale block where there are many,
// else less: span_grid), for several heads, K and V: finding the sequence and its pages costs a dozen
// dependent loads and integer divisions, which a warp a head would spend more time on than on its few
// KB.  Its warps go over the (K or V, head) pairs, neighbours at neighbouring heads, so that together
// they read whole rows.
// Sequence s owns the spans from first(s) / span + 2 s on: that is non-decreasing, leaves room for
// the spans that n tokens can touch (n / span + 2), and needs no prefix sum.
constexpr int kWarps = 8;
constexpr int kSpanShift = 6;

struct Span {
    int s;            // sequence
    KvSequence q;
    int64_t start;    // first position, a multiple of the span
    int lo, hi;       // the new tokens' positions in it
};

// False where this block has nothing to do.
__device__ __forceinline__ bool find_span(const KvArgs &a, int shift, Span &x) {
    auto begin = [&](int s) { return (int64_t)(__ldg(a.q_start + s) >> shift) + 2 * (int64_t)s; };
    x.s = find_and_check(a, blockIdx.x, threadIdx.x == 0 && blockIdx.y == 0, begin,
                         [](const KvSequence &q) { return q.length; });
    x.q = kv_sequence(a, x.s);
    if (!x.q.valid || x.q.count > x.q.length) return false;  // nothing of it is read or written
    const int64_t j = blockIdx.x - begin(x.s);
    if (j < 0 || x.q.count == 0) return false;
    const int p0 = x.q.length - x.q.count;
    x.start = ((int64_t)(p0 >> shift) + j) << shift;
    if (x.start >= x.q.length) return false;
    x.lo = max(p0, (int)x.start);
    x.hi = (int)min((int64_t)x.q.length, x.start + (1 << shift));
    return true;
}

__device__ __forceinline__ uint32_t max_bits(uint32_t m, const uint4 &v) {
    m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

// Four codes round(x * s) of two bf16 pairs: adding 1.5 * 2^23 rounds to an integer in the low byte.
// |x| <= g gives |x * s| < 127.5, so there is nothing to clip.
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float s) {
    const float2 magic = make_float2(12582912.f, 12582912.f);
    // scalar products: the packed ones may be fused with the sum, which then rounds only once
    const float2 u = __fadd2_rn(make_float2(__fmul_rn(__uint_as_float(a << 16), s),
                                            __fmul_rn(__uint_as_float(a & 0xFFFF0000u), s)), magic);
    const float2 v = __fadd2_rn(make_float2(__fmul_rn(__uint_as_float(b << 16), s),
                                            __fmul_rn(__uint_as_float(b & 0xFFFF0000u), s)), magic);
    return gather_low_bytes(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(v.x),
                            __float_as_uint(v.y));
}

__device__ __forceinline__ uint32_t recode4(uint32_t c, float r) {
    uint32_t d = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        d |= ((uint32_t)__float2int_rn(__fmul_rn((float)(int8_t)(c >> (8 * i)), r)) & 0xFFu) << (8 * i);
    return d;
}

// SMALL: scale blocks of 16 tokens, whose states stay in registers between the maximum and the
// codes; longer blocks do not fit there and are read twice (the second time from L1 or L2).
template <int D, bool SMALL>
__global__ void __launch_bounds__(32 * kWarps, 4)
    kv_append_kernel(KvArgs a, const uint8_t *__restrict__ K, int64_t ldk,
                     const uint8_t *__restrict__ V, int64_t ldv, int shift) {
    constexpr int LPT = D / 8;       // lanes a token: 16 bytes of bf16 each
    constexpr int TPW = 32 / LPT;    // tokens the warp reads at once
    constexpr int KEEP = SMALL ? 16 / TPW : 1;
    const int lane = threadIdx.x & 31;
    Span x;
    if (!find_span(a, shift, x)) return;
    const int block = 1 << a.block_shift;
    const int first = (x.lo - (int)x.start) >> a.block_shift;
    const int last = (x.hi - 1 - (int)x.start) >> a.block_shift;
    // page of block `lane` of the span (there are 1 .. 4)
    int page = -1;
    if (lane >= first && lane <= last) page = kv_page(a, x.s, (int)x.start + lane * block);
    const int sub = lane / LPT, off = lane % LPT;
    for (int pair = blockIdx.y * kWarps + (threadIdx.x >> 5); pair < 2 * a.kv_heads;
         pair += gridDim.y * kWarps) {
        const bool is_v = pair >= a.kv_heads;
        const int head = is_v ? pair - a.kv_heads : pair;
        const int64_t ld = 2 * (is_v ? ldv : ldk);  // bytes a token row
        for (int b = first; b <= last; ++b) {
            const int pg = __shfl_sync(0xFFFFFFFFu, page, b);
            if (pg < 0) continue;
            const int start = (int)x.start + b * block;
            const int lo = max(x.lo, start), hi = min(x.hi, start + block), count = hi - lo;
            int8_t *out = (is_v ? a.v_codes : a.k_codes) + kv_code_at(a, pg, head, start);
            float *step = (is_v ? a.v_scales : a.k_scales) + kv_scale_at(a, pg, head, start);
            const float d_old = lo > start ? *step : 0.f;
            const uint8_t *in = (is_v ? V : K) +
                                (int64_t)(x.q.first + lo - (x.q.length - x.q.count)) * ld + 2 * head * D;
            uint4 v[KEEP];
            uint32_t m = 0;
            if constexpr (SMALL) {
#pragma unroll
                for (int i = 0; i < KEEP; ++i) {
                    const int t = sub + i * TPW;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (t < count) v[i] = __ldg(reinterpret_cast<const uint4 *>(in + t * ld) + off);
                }
#pragma unroll
                for (int i = 0; i < KEEP; ++i) m = max_bits(m, v[i]);
            } else {
#pragma unroll 4
                for (int t = sub; t < count; t += TPW)
                    m = max_bits(m, __ldg(reinterpret_cast<const uint4 *>(in + t * ld) + off));
            }
            m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
            float mx = __uint_as_float(m << 16);
            if (mx < 1e-5f) mx = 1e-5f;  // keeps NaN
            const float g_old = __fmul_rn(127.f, d_old);
            const bool grown = !(mx <= g_old) && !isnan(g_old);
            const float g = grown ? mx : g_old;
            const float s8 = __fdiv_rn(127.f, g);
            if (grown && lo > start) {  // the block's older codes, with the new step
                const float r = __fmul_rn(d_old, s8);
                uint4 *old = reinterpret_cast<uint4 *>(out);
                for (int i = lane; i < (lo - start) * D / 16; i += 32) {
                    uint4 c = old[i];
                    c.x = recode4(c.x, r);
                    c.y = recode4(c.y, r);
                    c.z = recode4(c.z, r);
                    c.w = recode4(c.w, r);
                    old[i] = c;
                }
            }
            uint2 *dst = reinterpret_cast<uint2 *>(out + (lo - start) * D);
            if (!(g <= 3.4028235e38f)) {  // a NaN or infinite step: codes of 0, so that every
                                          // product with it is NaN
                for (int t = sub; t < count; t += TPW) dst[t * LPT + off] = make_uint2(0, 0);
            } else if constexpr (SMALL) {
#pragma unroll
                for (int i = 0; i < KEEP; ++i) {
                    const int t = sub + i * TPW;
                    if (t < count)
                        dst[t * LPT + off] = make_uint2(codes4(v[i].x, v[i].y, s8),
                                                        codes4(v[i].z, v[i].w, s8));
                }
            } else {
#pragma unroll 4
                for (int t = sub; t < count; t += TPW) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(in + t * ld) + off);
                    dst[t * LPT + off] = make_uint2(codes4(u.x, u.y, s8), codes4(u.z, u.w, s8));
                }
            }
            __syncwarp();  // every lane has read the old step
            if (lane == 0 && grown) *step = __fdiv_rn(g, 127.f);
        }
    }
}

// Four codes as two pairs of bf16 values.  The byte c xor 0x80 under 0x4B0000 is the float 2^23 + 128
// + c: one byte permutation and an exact subtraction (int to float conversions, 16 a clock and SM,
// kept half of the reading time busy).
__device__ __forceinline__ uint2 values4(uint32_t codes, float d) {
    const uint32_t u = codes ^ 0x80808080u;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = __fmul_rn(__uint_as_float(prmt(u, 0x4B000000u, 0x7540u + i)) - 8388736.f, d);
    return make_uint2(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]));
}

// Reads back a sequence's last tokens, 16 positions of one head at a time.  A scale block is at
// least 16 tokens, so the 16 share a step.
template <int D>
__global__ void __launch_bounds__(32 * kWarps, 6)
    kv_read_kernel(KvArgs a, uint8_t *__restrict__ K, int64_t ldk, uint8_t *__restrict__ V,
                   int64_t ldv, int shift) {
    constexpr int LPT = D / 8, TPW = 32 / LPT, N = kChunk / TPW;
    const int lane = threadIdx.x & 31;
    Span x;
    if (!find_span(a, shift, x)) return;
    const int first = (x.lo - (int)x.start) / kChunk, last = (x.hi - 1 - (int)x.start) / kChunk;
    int page = -1;  // of chunk `lane`
    if (lane >= first && lane <= last) page = kv_page(a, x.s, (int)x.start + lane * kChunk);
    const int sub = lane / LPT, off = lane % LPT;
    for (int pair = blockIdx.y * kWarps + (threadIdx.x >> 5); pair < 2 * a.kv_heads;
         pair += gridDim.y * kWarps) {
        const bool is_v = pair >= a.kv_heads;
        const int head = is_v ? pair - a.kv_heads : pair;
        const int64_t ld = 2 * (is_v ? ldv : ldk);
        for (int b = first; b <= last; ++b) {
            const int pg = __shfl_sync(0xFFFFFFFFu, page, b);
            if (pg < 0) continue;
            const int start = (int)x.start + b * kChunk;
            const uint2 *in = reinterpret_cast<const uint2 *>(
                (is_v ? a.v_codes : a.k_codes) + kv_code_at(a, pg, head, start));
            const float d = (is_v ? a.v_scales : a.k_scales)[kv_scale_at(a, pg, head, start)];
            uint8_t *out = (is_v ? V : K) + 2 * head * D +
                           (int64_t)(x.q.first + start - (x.q.length - x.q.count)) * ld;
            uint2 c[N];
#pragma unroll
            for (int i = 0; i < N; ++i) c[i] = __ldcs(in + 32 * i + lane);  // within the page
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int t = sub + i * TPW;
                if (start + t >= x.lo && start + t < x.hi) {
                    const uint2 lo = values4(c[i].x, d), hi = values4(c[i].y, d);
                    reinterpret_cast<uint4 *>(out + t * ld)[off] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
            }
        }
    }
}

}  // namespace

// The grid over spans and (K or V, head) pairs, a warp a pair: long spans where there are enough of
// them to fill the GPU (kFill blocks; read back of 44 000 tokens 52 us, 63 us with 16), else spans of
// one `shortest` (append of 8700 tokens 15 us, 25 us with 64); then the pairs are dealt to several
// blocks, up to three times kFill in all (those two 49 and 14 us).
constexpr int kFill = 4 * kSms;

static dim3 span_grid(const KvArgs &a, int shortest, int &shift) {
    auto spans = [&](int sh) { return ((int64_t)a.tokens >> sh) + 2 * (int64_t)a.batch; };
    shift = shortest < kSpanShift && spans(kSpanShift) < kFill ? shortest
                                                                : max(shortest, kSpanShift);
    const int64_t x = spans(shift), most = (2 * a.kv_heads + kWarps - 1) / kWarps;
    const int64_t y = (3 * kFill + x - 1) / x;
    return dim3((unsigned)x, (unsigned)(y < most ? y : most));
}

cudaError_t launch_kv_append(const KvArgs &a, const void *K, int64_t ldk, const void *V,
                             int64_t ldv, cudaStream_t stream) {
    int shift;
    const dim3 grid = span_grid(a, a.block_shift, shift);
    const bool small = a.block_shift == 4;
    auto kern = a.head_dim == 64 ? (small ? kv_append_kernel<64, true> : kv_append_kernel<64, false>)
                                 : (small ? kv_append_kernel<128, true> : kv_append_kernel<128, false>);
    kern<<<grid, 32 * kWarps, 0, stream>>>(a, static_cast<const uint8_t *>(K), ldk,
                                           static_cast<const uint8_t *>(V), ldv, shift);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvArgs &a, void *K, int64_t ldk, void *V, int64_t ldv,
                           cudaStream_t stream) {
    int shift;
    const dim3 grid = span_grid(a, 4, shift);  // 16 tokens: what a warp takes at once
    auto kern = a.head_dim == 64 ? kv_read_kernel<64> : kv_read_kernel<128>;
    kern<<<grid, 32 * kWarps, 0, stream>>>(a, static_cast<uint8_t *>(K), ldk,
                                           static_cast<uint8_t *>(V), ldv, shift);
    return cudaGetLastError();
}

}  // namespace bitnet
