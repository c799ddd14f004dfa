// kv_attention.cu -- attention of a few new tokens over the paged 8-bit K/V cache (decoding), and
// the choice between this kernel and the one for prompts (kv_attention_tc.cu).
//
// For a new token at position p of its sequence and query head h of the key head's group:
//   s_t = scale * d_K(t) * (q . c_K(t)),  t <= p (causal) or t < length
//   y   = sum_t exp(s_t) d_V(t) c_V(t) / sum_t exp(s_t),   lse = log sum_t exp(s_t)
// With few rows a code is used once or a few times, so the kernel is bound by the stream of codes
// from HBM: 23 codes per SM and clock at the measured copy rate, which leaves each code about five
// lane instructions.
//
// Rows.  The new tokens of a sequence times the query heads of one key head, in tiles of 8 * NT (one
// of 8, or up to two of 16 whose blocks are neighbours and meet in L2); a tile's rows share every
// load and conversion of a code.  The products run as
//   S^T [16 tokens x 8 rows] = K [16 x D] Q^T,   O^T [D x 8 rows] += V^T [D x 16] W^T
// with mma.m16n8k16, the codes as the 16-row operand: the 8-column operand then wastes little on
// the rows that are not there.  (tcgen05 would need the converted codes in shared memory: 1 + 1
// bytes to bring them there and read them, 2 + 2 to write and read the fp16 ones, 6 x 23 bytes a
// clock, above the 128 that shared memory moves; here it is 2 x 23.)
//
// Codes to fp16.  A code c of -128 .. 127 xor 0x80 is the byte c + 128; under the byte 0x64 that is
// the fp16 number 1152 + c, and one subtraction gives c exactly.  q is scaled by a power of two a
// row (row_scaling), so bf16 -> fp16 loses only bits below 2^-38 of the row's largest; products are exact and
// summed in fp32.  The order of the features inside an mma's k is free, so a lane takes 16
// consecutive codes of a token with one 16-byte read.
//
// Weights.  d_V varies from block to block, so it belongs to the weight: w_t = exp2(s_t log2 e +
// log2 d_V(t) - m), m a reference that follows the row's maximum of that sum.  w is rounded to fp16
// for the product with the codes; the denominator sums w_t / d_V(t) in fp32, unrounded.  A block is
// at least 16 tokens, so a chunk of 16 has one d_K and one d_V.
// fp16 has 16 binary orders above 1 and 25 below, where a weight that is too small vanishes from the
// numerator: m is put 7 below the maximum, so the row's largest weight is in (2^6, 2^7] and one of
// 2^-31 of it is still seen (a token that takes nearly all of the weight, in front of a long cache:
// with the maximum at 1 the output was several per cent off).  m is only moved when a chunk exceeds 2^15:
// nearly all chunks need one vote instead of a reduction and a rescaling.  It moves by whole numbers,
// so rescaling is exact.
//
// Work split.  Per key head the chunks of all sequences form one line, cut into equal ranges, one
// for each of P blocks (P * heads fills the SMs once): ragged batches, single long sequences and
// many short ones all end together.  The ranges are computed from kv_len on the device, so a
// replayed graph follows its lengths.  A block whose range covers a sequence writes the output;
// of a sequence that several share, each writes its sums (at most its first and its last piece:
// two places a block), and a second kernel joins them in a fixed order.
//
// In a block each of eight warps takes every eighth chunk through its own ring of stages, filled
// with cp.async (16 bytes a lane) into an xor-swizzled layout: no barrier between the warps, and
// both kinds of 16-byte reads are free of bank conflicts.
//
// Measured on B200 (D = 128, 32 ragged sequences of 2000 .. 8000 tokens, 8 key heads, 334 MB): 4 rows
// 68 us, 8 rows 71 us, 16 rows 95 us, 32 rows 170 us (the tensor-core kernel: 240 us, so it takes
// over above 32); one sequence of 131072 tokens, 4 rows, 57 us.  The stream runs at 5.7 TB/s
// behind about 12 us of launch, dependent loads (lengths, page, codes), last chunks and join.
#include "kv_common.cuh"

namespace bitnet {
namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr float kTop = 7.f;     // log2 of where a moved reference puts the largest weight, and of
constexpr float kLimit = 15.f;  // the weight above which it moves
constexpr int kMinChunks = 32;  // shorter ranges do not repay the second launch (about 4 us)

// The device's view of the partial sums: [2 * P][heads][rows][D] sums, then [..][rows][2] maxima
// and denominators, then one int4 a block: what to join behind it.
struct Parts {
    float *sums, *stats;
    int4 *joins;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// Where the 16-byte piece `c` of token `t` (0 .. 15) lies in a chunk of codes: xor-swizzled so that
// neither the reads of K (8 lanes: 2 tokens x 4 pieces) nor those of V (8 lanes: 4 tokens x 2
// pieces; D = 64: 16 lanes of 8 bytes) meet in a bank.
template <int D>
__device__ __forceinline__ uint32_t piece(int t, int c) {
    if constexpr (D == 128) {
        const int f = ((t & 4) ^ ((t & 1) << 2)) | (t & 2);
        return (uint32_t)(t * 8 + (c ^ f)) * 16;
    } else {
        const int line = t >> 1, slot = (((t & 1) << 2) | c) ^ (2 * (line & 3));
        return (uint32_t)(line * 8 + slot) * 16;
    }
}

__device__ __forceinline__ int chunks_of(int length) {
    return length > 0 ? (length + kChunk - 1) / kChunk : 1;  // an empty sequence still has outputs
}

// The length that takes part: 0 for a sequence that is left out.
__device__ __forceinline__ int work_length(const KvArgs &a, const AttentionArgs &at, int s) {
    const KvSequence q = kv_sequence(a, s);
    return q.valid && q.count > 0 && q.count <= at.max_new ? q.length : 0;
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 2 : 1)
    kv_attention_kernel(KvArgs a, AttentionArgs at, Parts parts, int P, int RT) {
    constexpr int ROWS = 8 * NT;
    constexpr int CB = kChunk * D;           // bytes of a chunk of codes
    constexpr int STAGE = 2 * CB + 16;       // K, V and their steps
    constexpr int KW = D / 16;               // 4-code words of a token a lane holds = k16 steps
    constexpr int MT = D / 16;               // 16-feature tiles of O^T
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red_m[kWarps][ROWS], red_l[kWarps][ROWS];
    __shared__ long long scan[kWarps];
    __shared__ int found[4];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane >> 2, t = lane & 3;
    // a group of rows: a key head, and one of RT tiles of ROWS rows (neighbours share the codes in L2)
    const int p = blockIdx.x / (a.kv_heads * RT), group = blockIdx.x - p * a.kv_heads * RT;
    const int head = group / RT, row0 = (group - head * RT) * ROWS;
    const int G = at.q_heads / a.kv_heads;
    pdl_wait();  // lengths, queries and codes come from the kernels before
    pdl_launch_dependents();

    // ---- this block's range of the line of chunks ----
    // each thread counts a run of sequences; a scan over the threads gives the total and the first
    // sequence of the range
    const int run = (a.batch + 32 * kWarps - 1) / (32 * kWarps);
    const int run0 = min(tid * run, a.batch), run1 = min(run0 + run, a.batch);
    long long mine = 0;
    for (int s = run0; s < run1; ++s) mine += chunks_of(work_length(a, at, s));
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    long long total = 0, base = upto - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += scan[w];
        total += scan[w];
    }
    const long long workers = min((long long)P, (total + kMinChunks - 1) / kMinChunks);
    const long long quota = (total + workers - 1) / workers;
    const long long t0 = p * quota, t1 = min(t0 + quota, total);
    if (t0 >= t1) {  // nothing left for this block
        if (group == 0 && tid == 0 && P > 1) parts.joins[p] = make_int4(-1, 0, 0, 0);
        return;
    }
    if (mine > 0 && base <= t0 && t0 < base + mine) {
        int s = run0;
        for (;; ++s) {
            const int c = chunks_of(work_length(a, at, s));
            if (t0 < base + c) break;
            base += c;
        }
        found[0] = s;
        found[1] = (int)(t0 - base);
    }
    __syncthreads();
    int s = found[0], c0 = found[1];
    long long at_chunk = t0;  // line position of chunk c0 of sequence s
    if (group == 0 && tid == 0 && P > 1) parts.joins[p] = make_int4(-1, 0, 0, 0);

    const uint32_t ring = smem_addr(smem) + warp * kStages * STAGE;
    const int code_shift = a.page_shift + (D == 128 ? 7 : 6), scale_shift = a.page_shift - a.block_shift;
    const float *my_scales = lane ? a.v_scales : a.k_scales;
    // this lane's places in a stage: of the pieces it brings (and, for D = 128, four tokens on), of
    // its first piece of K, of its pieces of V of an even and an odd token
    const uint32_t to_even = piece<D>(lane / (D / 16), lane % (D / 16));
    const uint32_t to_odd = piece<D>(lane / (D / 16) + 4, lane % (D / 16));
    const uint32_t k_piece = piece<D>(n, t);
    const uint32_t v_even = D == 128 ? piece<D>(2 * t, n) : piece<D>(2 * t, n >> 1) + (n & 1) * 8;
    const uint32_t v_odd = D == 128 ? piece<D>(2 * t + 1, n) : piece<D>(2 * t + 1, n >> 1) + (n & 1) * 8;
    while (at_chunk < t1) {
        const KvSequence q = kv_sequence(a, s);
        const bool out_of_use = !q.valid || q.count > at.max_new;
        if (out_of_use && tid == 0) record_status(a.status, BITNET_ERR_INVALID);
        const int length = out_of_use || q.count == 0 ? 0 : q.length;
        const int rows = out_of_use ? 0 : min(q.count * G - row0, ROWS);  // of this tile
        const int chunks = chunks_of(length);
        const int c1 = (int)min((long long)chunks, c0 + (t1 - at_chunk));
        // an empty sequence's one chunk is not there; a tile without rows reads nothing
        const int real = length > 0 && rows > 0 ? c1 : c0;

        // ---- the ring ----
        const int first = c0 + warp;
        const int count = real > first ? (real - first + kWarps - 1) / kWarps : 0;
        const int32_t *table = a.page_table + (int64_t)s * a.max_pages;
        int page = count > 0 ? table[first * kChunk >> a.page_shift] : 0;  // of the next
        int bring_pos = first * kChunk, left = count;                                 // chunk
        uint32_t bring_to = ring;
        uint32_t no_page = 0;  // bit k: the chunk that was asked for k calls ago has no page
        auto bring = [&]() {
            no_page <<= 1;
            if (left > 0) {
                if ((uint32_t)page < (uint32_t)a.num_pages) {
                    const int in_page = bring_pos & ((1 << a.page_shift) - 1);
                    const int64_t tile = (int64_t)page * a.kv_heads + head;
                    const int64_t at_code = (tile << code_shift) + (in_page * D + 16 * lane);
                    const int8_t *ks = a.k_codes + at_code, *vs = a.v_codes + at_code;
#pragma unroll
                    for (int i = 0; i < CB / 512; ++i) {  // 512 bytes on: D = 128: 4 tokens, D = 64: 8
                        const uint32_t d = bring_to + (D == 128 && (i & 1) ? to_odd : to_even) +
                                           (D == 128 ? (i >> 1) * 1024 : i * 512);
                        cp_async16(d, ks + 512 * i);
                        cp_async16(d + CB, vs + 512 * i);
                    }
                    if (lane < 2)
                        cp_async4(bring_to + 2 * CB + 4 * lane,
                                  my_scales + (tile << scale_shift) + (in_page >> a.block_shift));
                } else {
                    record_status(a.status, BITNET_ERR_INVALID);
                    no_page |= 1;
                }
                --left;
                bring_pos += kWarps * kChunk;
                bring_to = bring_to == ring + (kStages - 1) * STAGE ? ring : bring_to + STAGE;
                if (left > 0) page = table[bring_pos >> a.page_shift];
            }
            cp_async_commit();
        };
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) bring();
        // ---- Q: this lane's features of row n (and n + 8), scaled as fp16 ----
        uint32_t qf[NT][2 * KW];
        float rowf[NT][2];  // scale * log2 e / that scaling, rows 2t and 2t + 1
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int r = 8 * i + n;
            uint2 w[KW];
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < KW; ++j) w[j] = make_uint2(0, 0);
            if (r < rows) {
                const uint8_t *src = static_cast<const uint8_t *>(at.Q) +
                                     2 * ((int64_t)(q.first + (row0 + r) / G) * at.ldq +
                                          (int64_t)(head * G + (row0 + r) % G) * D);
#pragma unroll
                for (int j = 0; j < KW / 4; ++j) {
                    const uint4 *v = reinterpret_cast<const uint4 *>(src + 32 * (t + 4 * j));
                    const uint4 x = v[0], y = v[1];
                    w[4 * j] = make_uint2(x.x, x.y);
                    w[4 * j + 1] = make_uint2(x.z, x.w);
                    w[4 * j + 2] = make_uint2(y.x, y.y);
                    w[4 * j + 3] = make_uint2(y.z, y.w);
                }
            }
#pragma unroll
            for (int j = 0; j < KW; ++j)
                mx = __vmaxu2(__vmaxu2(mx, w[j].x & 0x7FFF7FFFu), w[j].y & 0x7FFF7FFFu);
            mx = max(mx & 0xFFFFu, mx >> 16);
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            float up, down;
            row_scaling(mx, down, up);
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                qf[i][2 * j] = half2_of(__uint_as_float(w[j].x << 16) * down,
                                        __uint_as_float(w[j].x & 0xFFFF0000u) * down);
                qf[i][2 * j + 1] = half2_of(__uint_as_float(w[j].y << 16) * down,
                                            __uint_as_float(w[j].y & 0xFFFF0000u) * down);
            }
            const float f = up * (at.scale * kLog2e);
            rowf[i][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * t);
            rowf[i][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * t + 4);
        }
        // what rows 2t, 2t + 1 see; rows that are not there see everything and are dropped
        int seen[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 8 * i + 2 * t + k;
                seen[i][k] = at.causal && r < rows ? length - q.count + (row0 + r) / G + 1 : length;
            }
        const int all_see = at.causal ? length - q.count + row0 / G + 1 : length;

        float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            m[i][0] = m[i][1] = kNothing;
            l[i][0] = l[i][1] = 0.f;
#pragma unroll
            for (int j = 0; j < MT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
        }

        uint32_t stage = ring;
        int pos = first * kChunk;
        for (int k = 0; k < count; ++k) {
            bring();
            cp_async_wait<kStages - 1>();
            __syncwarp();
            if (!(no_page >> (kStages - 1) & 1)) {  // tokens of no page weigh nothing
                const uint2 step2 = lds64(stage + 2 * CB);
                const float dk = __uint_as_float(step2.x), dv = v_step(__uint_as_float(step2.y));
                float sc[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
                // S^T: tokens n and n + 8
#pragma unroll
                for (int j = 0; j < KW / 4; ++j) {
                    const uint4 x = lds128(stage + (k_piece ^ (64 * j)));
                    const uint4 y = lds128(stage + (k_piece ^ (64 * j)) + CB / 2);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t u = xs[e] ^ 0x80808080u, v = ys[e] ^ 0x80808080u;
                        const uint32_t a0 = codes_lo(u), a1 = codes_lo(v), a2 = codes_hi(u),
                                       a3 = codes_hi(v);
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            mma_f16(sc[i], a0, a1, a2, a3, qf[i][2 * (4 * j + e)],
                                    qf[i][2 * (4 * j + e) + 1]);
                    }
                }
                // V, already on its way while the weights are made
                uint32_t vw[4][MT / 2];
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
                    const uint32_t from = stage + CB + (e & 1 ? v_odd : v_even) + (e >> 1) * (CB / 2);
                    if constexpr (D == 128) {
                        const uint4 x = lds128(from);
                        vw[e][0] = x.x; vw[e][1] = x.y; vw[e][2] = x.z; vw[e][3] = x.w;
                    } else {
                        const uint2 x = lds64(from);
                        vw[e][0] = x.x; vw[e][1] = x.y;
                    }
                }
                // weights
                const float lv = log2_approx(dv), rv = rcp_approx(dv);
                uint32_t wt[NT][2];
                bool over = false;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float f0 = rowf[i][0] * dk, f1 = rowf[i][1] * dk;
                    sc[i][0] = fmaf(sc[i][0], f0, lv);
                    sc[i][1] = fmaf(sc[i][1], f1, lv);
                    sc[i][2] = fmaf(sc[i][2], f0, lv);
                    sc[i][3] = fmaf(sc[i][3], f1, lv);
                    if (pos + kChunk > all_see) {
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4)
                            if (pos + n + 8 * (k4 >> 1) >= seen[i][k4 & 1]) sc[i][k4] = -INFINITY;
                    }
                    over |= fmaxf(sc[i][0], sc[i][2]) > m[i][0] + kLimit ||
                            fmaxf(sc[i][1], sc[i][3]) > m[i][1] + kLimit;
                }
                if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2) {
                            float x = fmaxf(sc[i][k2], sc[i][k2 + 2]);
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                            x = fmaxf(ceilf(x) - kTop, m[i][k2]);
                            const float keep = exp2_approx(m[i][k2] - x);
                            m[i][k2] = x;
                            l[i][k2] *= keep;
#pragma unroll
                            for (int j = 0; j < MT; ++j) {
                                o[i][j][k2] *= keep;
                                o[i][j][k2 + 2] *= keep;
                            }
                        }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float w0 = exp2_approx(sc[i][0] - m[i][0]), w1 = exp2_approx(sc[i][1] - m[i][1]);
                    const float w2 = exp2_approx(sc[i][2] - m[i][0]), w3 = exp2_approx(sc[i][3] - m[i][1]);
                    const float s0 = w0 + w2, s1 = w1 + w3;
                    // a row that sees none of the chunk takes nothing of it, whatever its step is
                    if (s0 != 0.f) l[i][0] = fmaf(s0, rv, l[i][0]);
                    if (s1 != 0.f) l[i][1] = fmaf(s1, rv, l[i][1]);
                    wt[i][0] = transpose8x8(half2_of(w0, w1));
                    wt[i][1] = transpose8x8(half2_of(w2, w3));
                }
                // O^T += V^T W^T: this lane's features are d = (D / 8) n + 2j (+ 1)
#pragma unroll
                for (int e = 0; e < MT / 2; ++e) {
                    uint32_t f[2][4];  // [token pair][feature 4e ..]
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u = vw[2 * h][e] ^ 0x80808080u;
                        const uint32_t v = vw[2 * h + 1][e] ^ 0x80808080u;
                        const uint32_t x = prmt(u, v, 0x5140u), y = prmt(u, v, 0x7362u);
                        f[h][0] = codes_lo(x);
                        f[h][1] = codes_hi(x);
                        f[h][2] = codes_lo(y);
                        f[h][3] = codes_hi(y);
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        mma_f16(o[i][2 * e], f[0][0], f[0][1], f[1][0], f[1][1], wt[i][0], wt[i][1]);
                        mma_f16(o[i][2 * e + 1], f[0][2], f[0][3], f[1][2], f[1][3], wt[i][0],
                                wt[i][1]);
                    }
                }
            }
            __syncwarp();  // the stage may be filled again
            stage = stage == ring + (kStages - 1) * STAGE ? ring : stage + STAGE;
            pos += kWarps * kChunk;
        }

        // ---- join the warps ----
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                l[i][k] += __shfl_xor_sync(0xFFFFFFFFu, l[i][k], 4);
                l[i][k] += __shfl_xor_sync(0xFFFFFFFFu, l[i][k], 8);
                l[i][k] += __shfl_xor_sync(0xFFFFFFFFu, l[i][k], 16);
                if (n == 0) {
                    red_m[warp][8 * i + 2 * t + k] = m[i][k];
                    red_l[warp][8 * i + 2 * t + k] = l[i][k];
                }
            }
        cp_async_wait<0>();
        __syncthreads();  // every warp has left its ring: it holds the sums now
        float *acc = reinterpret_cast<float *>(smem);  // [warp][row][D + 4]
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float *dst = acc + ((warp * ROWS + 8 * i + 2 * t + k) * (D + 4)) + n * (D / 8);
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    *reinterpret_cast<float2 *>(dst + 2 * j) = make_float2(o[i][j][k], o[i][j][k + 2]);
            }
        __syncthreads();
        const bool whole = c0 == 0 && c1 == chunks;
        const int slot = 2 * p + (at_chunk != t0);
        for (int x = tid; x < rows * (D / 4); x += 32 * kWarps) {
            const int r = x / (D / 4), d = (x - r * (D / 4)) * 4;
            float mr = kNothing;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mr = fmaxf(mr, red_m[w][r]);
            float lr = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float keep = exp2_approx(red_m[w][r] - mr);
                const float4 u = *reinterpret_cast<const float4 *>(acc + (w * ROWS + r) * (D + 4) + d);
                lr = fmaf(red_l[w][r], keep, lr);
                v.x = fmaf(u.x, keep, v.x);
                v.y = fmaf(u.y, keep, v.y);
                v.z = fmaf(u.z, keep, v.z);
                v.w = fmaf(u.w, keep, v.w);
            }
            if (whole) {
                const float inv = lr == 0.f ? 0.f : __fdividef(1.f, lr);
                const int64_t token = q.first + (row0 + r) / G, qh = head * G + (row0 + r) % G;
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(at.Y) +
                                           2 * (token * at.ldy + qh * D + d)) =
                    make_uint2(bf16x2_of(v.x * inv, v.y * inv), bf16x2_of(v.z * inv, v.w * inv));
                if (at.lse && d == 0)
                    at.lse[token * at.q_heads + qh] =
                        lr == 0.f ? -INFINITY : (mr + log2_approx(lr)) * kLn2;
            } else {
                const int64_t row = ((int64_t)slot * a.kv_heads * RT + group) * ROWS + r;
                *reinterpret_cast<float4 *>(parts.sums + row * D + d) = v;
                if (d == 0) *reinterpret_cast<float2 *>(parts.stats + 2 * row) = make_float2(mr, lr);
            }
        }
        // a sequence that begins in this range and ends in a later one is joined behind this block
        if (group == 0 && tid == 0 && c0 == 0 && c1 < chunks)
            parts.joins[p] = make_int4(s, (int)((at_chunk + chunks - 1) / quota) - p + 1, slot, 0);
        __syncthreads();  // the sums have been read: the ring may be filled again
        at_chunk += c1 - c0;
        c0 = 0;
        ++s;
    }
}

// Joins the pieces of the sequence that begins in the range of block p and ends in a later one:
// four rows of one key head at a time, four warps each, the pieces in turn.  (Most blocks have
// nothing to join; with eight rows at a time starting them took 2 us more.)
constexpr int kJoinRows = 4;

template <int D, int NT>
__global__ void __launch_bounds__(128 * kJoinRows)
    kv_attention_join_kernel(KvArgs a, AttentionArgs at, Parts parts, int P, int RT) {
    constexpr int F = D / 32;  // features a lane
    __shared__ float sums[kJoinRows][3][D], stats[kJoinRows][3][2];
    pdl_launch_dependents();
    pdl_wait();
    const int p = blockIdx.x % P, group = blockIdx.x / P, head = group / RT;
    const int row0 = (group - head * RT) * 8 * NT;
    const int4 join = parts.joins[p];
    if (join.x < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3;
    const KvSequence q = kv_sequence(a, join.x);
    const int G = at.q_heads / a.kv_heads, rows = min(q.count * G - row0, 8 * NT);
    for (int r0 = 0; r0 < rows; r0 += kJoinRows) {
        const int r = r0 + (warp >> 2);
        const bool live = r < rows;
        float m = kNothing, l = 0.f, v[F] = {};
        if (live) {
#pragma unroll 4
            for (int i = quarter; i < join.y; i += 4) {
                const int64_t slot = i == 0 ? join.z : 2 * (p + i);
                const int64_t row = (slot * a.kv_heads * RT + group) * (8 * NT) + r;
                const float2 ml = *reinterpret_cast<const float2 *>(parts.stats + 2 * row);
                float u[F];
                if constexpr (F == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(parts.sums + row * D + 4 * lane);
                    u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(parts.sums + row * D + 2 * lane);
                    u[0] = x.x; u[1] = x.y;
                }
                const float mn = fmaxf(m, ml.x);
                const float old = exp2_approx(m - mn), now = exp2_approx(ml.x - mn);
                l = l * old + ml.y * now;
#pragma unroll
                for (int f = 0; f < F; ++f) v[f] = v[f] * old + u[f] * now;
                m = mn;
            }
        }
        if (live && quarter) {
            for (int f = 0; f < F; ++f) sums[warp >> 2][quarter - 1][F * lane + f] = v[f];
            if (lane == 0) {
                stats[warp >> 2][quarter - 1][0] = m;
                stats[warp >> 2][quarter - 1][1] = l;
            }
        }
        __syncthreads();
        if (live && quarter == 0) {
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const float mi = stats[warp >> 2][i][0], li = stats[warp >> 2][i][1];
                const float mn = fmaxf(m, mi);
                const float old = exp2_approx(m - mn), now = exp2_approx(mi - mn);
                l = l * old + li * now;
#pragma unroll
                for (int f = 0; f < F; ++f)
                    v[f] = v[f] * old + sums[warp >> 2][i][F * lane + f] * now;
                m = mn;
            }
            const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
            const int64_t token = q.first + (row0 + r) / G, qh = head * G + (row0 + r) % G;
            uint8_t *Y = static_cast<uint8_t *>(at.Y) + 2 * (token * at.ldy + qh * D + F * lane);
            uint32_t y[F / 2];
#pragma unroll
            for (int f = 0; f < F / 2; ++f)
                y[f] = bf16x2_of(v[2 * f] * inv, v[2 * f + 1] * inv);
            if constexpr (F == 4)
                *reinterpret_cast<uint2 *>(Y) = make_uint2(y[0], y[1]);
            else
                *reinterpret_cast<uint32_t *>(Y) = y[0];
            if (at.lse && lane == 0)
                at.lse[token * at.q_heads + qh] = l == 0.f ? -INFINITY : (m + log2_approx(l)) * kLn2;
        }
        __syncthreads();
    }
}

// How the rows of a sequence and key head are cut: RT tiles of 8 * nt rows; nt 0 for the other kernel.
struct RowTiles {
    int nt, RT;
};
RowTiles row_tiles(const KvArgs &a, const AttentionArgs &at) {
    const int64_t rows = (int64_t)at.max_new * (at.q_heads / a.kv_heads);
    if (rows > kDecodeRows) return {0, 0};
    return rows <= 8 ? RowTiles{1, 1} : RowTiles{2, (int)(rows + 15) / 16};
}

// Blocks per key head and row tile: as many as fill the SMs, no more than the longest batch that the
// page table allows can use.
int worker_blocks(const KvArgs &a, RowTiles t) {
    const int64_t fill = kSms * (t.nt == 1 ? 2 : 1) / (a.kv_heads * t.RT);
    const int64_t most = ((int64_t)a.batch * ((int64_t)a.max_pages << a.page_shift) / kChunk +
                          a.batch + kMinChunks - 1) / kMinChunks;
    const int64_t p = fill < most ? fill : most;
    return p < 1 ? 1 : (int)p;
}

size_t part_rows(const KvArgs &a, RowTiles t, int P) {  // rows of partial sums
    return (size_t)2 * P * a.kv_heads * t.RT * 8 * t.nt;
}

template <int D, int NT>
cudaError_t launch_decode(const KvArgs &a, const AttentionArgs &at, void *ws, cudaStream_t stream,
                          int *launches) {
    const RowTiles t = row_tiles(a, at);
    const int P = worker_blocks(a, t);
    constexpr int ring = kWarps * kStages * (2 * kChunk * D + 16);
    constexpr int join = kWarps * 8 * NT * (D + 4) * 4;
    constexpr int smem = ring > join ? ring : join;
    Parts parts = {};
    if (P > 1) {
        const size_t rows = part_rows(a, t, P);
        parts.sums = static_cast<float *>(ws);
        parts.stats = parts.sums + rows * D;
        parts.joins = reinterpret_cast<int4 *>(parts.stats + rows * 2);
    }
    auto kern = kv_attention_kernel<D, NT>;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const unsigned grid = (unsigned)(P * a.kv_heads * t.RT);
    // Programmatic launches: both kernels are set up while the one before them ends, and wait for it
    // before they read anything (calls one after the other: 72.8 -> 69.9 us on the ragged batch).
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *launches = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, at, parts, P, t.RT);
    if (e != cudaSuccess || P == 1) return e;
    cfg.blockDim = dim3(128 * kJoinRows);
    cfg.dynamicSmemBytes = 0;
    *launches = 2;
    return cudaLaunchKernelEx(&cfg, kv_attention_join_kernel<D, NT>, a, at, parts, P, t.RT);
}

}  // namespace

size_t kv_attention_workspace(const KvArgs &a, const AttentionArgs &at) {
    const RowTiles t = row_tiles(a, at);
    if (t.nt == 0) return kv_attention_tc_workspace(a, at);
    const int P = worker_blocks(a, t);
    return P == 1 ? 0 : part_rows(a, t, P) * (a.head_dim + 2) * 4 + (size_t)P * sizeof(int4);
}

cudaError_t launch_kv_attention(const KvArgs &a, const AttentionArgs &at, void *ws,
                                cudaStream_t stream, int *launches) {
    switch (row_tiles(a, at).nt) {
        case 1:
            return a.head_dim == 64 ? launch_decode<64, 1>(a, at, ws, stream, launches)
                                    : launch_decode<128, 1>(a, at, ws, stream, launches);
        case 2:
            return a.head_dim == 64 ? launch_decode<64, 2>(a, at, ws, stream, launches)
                                    : launch_decode<128, 2>(a, at, ws, stream, launches);
    }
    return launch_kv_attention_tc(a, at, ws, stream, launches);
}

}  // namespace bitnet
