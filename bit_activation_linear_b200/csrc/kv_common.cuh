// kv_common.cuh -- what the kernels on the paged 8-bit K/V cache share: the view they are given,
// and how they find the sequence that a piece of work belongs to.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace bitnet {

// The largest s in [0, batch) with begin(s) <= w, by one warp: every step probes 32 places, so a
// batch of 1024 takes two steps.  begin() is non-decreasing for valid input; whatever it returns,
// the result is in range (batch >= 1).
template <class F>
__device__ __forceinline__ int find_sequence(int64_t w, int batch, F &&begin) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = batch;
    while (len > 1) {
        const int step = (len + 31) / 32, at = lane * step;
        const bool before = at < len && (at == 0 || begin(lo + at) <= w);
        const int hits = __popc(__ballot_sync(0xFFFFFFFFu, before));
        const int skip = (hits - 1) * step;
        lo += skip;
        len = min(step, len - skip);
    }
    return lo;
}

// Rows of one sequence among the packed new tokens, and its cached length.
struct KvSequence {
    int first, count, length;  // rows [first, first + count); the length counts them
    bool valid;
};

__device__ __forceinline__ KvSequence kv_sequence_of(const KvArgs &a, int b, int e, int length) {
    KvSequence q;
    q.first = b;
    q.length = length;
    q.valid = b >= 0 && e >= b && e <= a.tokens && q.length >= 0 &&
              (int64_t)q.length <= (int64_t)a.max_pages << a.page_shift;
    q.count = q.valid ? e - b : 0;
    return q;
}

// (No __ldg here, in kv_page_entry and in the streaming kernel, which is launched programmatically: it
// runs, up to its pdl_wait(), beside the kernel that may be writing these; see ld_written in common.cuh.)
__device__ __forceinline__ KvSequence kv_sequence(const KvArgs &a, int s) {
    return kv_sequence_of(a, a.q_start[s], a.q_start[s + 1], a.kv_len[s]);
}

// The sequence of piece w of the work, found with find_sequence.  Where q_start goes back, a piece
// may find another sequence than its own, so the pieces that find a sequence cannot answer for it
// being reported: piece w also looks at sequence w (there are more pieces than sequences) if `look`,
// and records one that is not valid or has more new tokens than most(sequence).  Its loads are asked
// for in front of the search and looked at behind it.
template <class F, class G>
__device__ __forceinline__ int find_and_check(const KvArgs &a, int64_t w, bool look, F &&begin,
                                              G &&most) {
    int b = 0, e = 0, length = 0;
    look = look && w < a.batch;
    if (look) {
        b = __ldg(a.q_start + w);
        e = __ldg(a.q_start + w + 1);
        length = __ldg(a.kv_len + w);
    }
    const int s = find_sequence(w, a.batch, begin);
    if (look) {
        const KvSequence q = kv_sequence_of(a, b, e, length);
        if (!q.valid || q.count > most(q)) record_status(a.status, BITNET_ERR_INVALID);
    }
    return s;
}

// Page that holds `position` of sequence s, or -1 (recorded as an invalid argument); the entry of
// the page table and its check apart, for kernels that ask for it ahead of its use.
__device__ __forceinline__ int kv_page_entry(const KvArgs &a, int s, int position) {
    return a.page_table[(int64_t)s * a.max_pages + (position >> a.page_shift)];
}
__device__ __forceinline__ int kv_page_checked(const KvArgs &a, int page) {
    if (page < 0 || page >= a.num_pages) {
        record_status(a.status, BITNET_ERR_INVALID);
        return -1;
    }
    return page;
}
__device__ __forceinline__ int kv_page(const KvArgs &a, int s, int position) {
    return kv_page_checked(a, kv_page_entry(a, s, position));
}

// Codes of a position in a page, and the step of its block.
__device__ __forceinline__ int64_t kv_code_at(const KvArgs &a, int page, int head, int position) {
    const int in_page = position & ((1 << a.page_shift) - 1);
    return ((((int64_t)page * a.kv_heads + head) << a.page_shift) + in_page) * a.head_dim;
}

__device__ __forceinline__ int64_t kv_scale_at(const KvArgs &a, int page, int head, int position) {
    const int in_page = position & ((1 << a.page_shift) - 1);
    return (((int64_t)page * a.kv_heads + head) << (a.page_shift - a.block_shift)) +
           (in_page >> a.block_shift);
}

// ------------------------------------------------------------------------------------------
// What the attention kernels share
// ------------------------------------------------------------------------------------------
constexpr int kChunk = 16;      // tokens: a scale block is a whole number of chunks
// The SMs that splits are made for: a constant, because the workspace query answers without a device
// and the launch has to come to the same split.
constexpr int kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNothing = -3.0e38f;  // the reference of a row that has seen nothing
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t sub_1152(uint32_t two) {
    uint32_t d;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(d) : "r"(two), "r"(0x64806480u));
    return d;
}
// Bytes 0 and 1, or 2 and 3, of c + 128 as two fp16 numbers c.
__device__ __forceinline__ uint32_t codes_lo(uint32_t u) { return sub_1152(prmt(u, 0x64646464u, 0x4140u)); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t u) { return sub_1152(prmt(u, 0x64646464u, 0x4342u)); }

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float2 float2_of(uint32_t two) {
    float2 d;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}" : "=f"(d.x), "=f"(d.y) : "r"(two));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// bf16 pairs of a row of Q (largest magnitude `mx` as bf16 bits): the powers of two that scale it to
// below 2^15, under fp16's limit, and back.  The row's features then keep their bits down to 2^-38 of
// its largest (scaled to below 2 they kept 2^-24: where a large feature meets zeros in the keys, the
// scores are made of the small ones).  Rows below 2^-62 are scaled to below 2, so that `up` and the
// products with it stay normal numbers; 1 for zeros, infinities and NaN (the outputs of a row that
// has one are NaN).
__device__ __forceinline__ void row_scaling(uint32_t mx, float &down, float &up) {
    const uint32_t ex = mx >> 7, at = ex > 64 ? ex - 14 : max(ex, 1u);
    up = mx != 0 && ex < 255 ? __uint_as_float(at << 23) : 1.f;
    down = 1.f / up;
}

// d_V as the weights carry it: never 0 (a log2 is taken of it), NaN and infinity as they are.  The
// denominator sums weights of up to 2^15 over d_V: with 2^-90 it stays below 2^126, from where the
// fast division gives 0, for 2^21 tokens.
__device__ __forceinline__ float v_step(float d) { return d < 8e-28f ? 8e-28f : d; }

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

}  // namespace bitnet
