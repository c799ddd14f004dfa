// kv_attention_tc.cu -- attention of prompts (more than 32 rows a sequence and key head) over the
// paged 8-bit K/V cache, on the tensor cores.  The formulas, the way codes become fp16 and the way
// d_V goes into the weights are those of kv_attention.cu.
//
// A block takes 256 rows (new token, query head of the group) of one sequence and key head as two
// tiles of 128, and walks the cache in steps of 128 tokens:
//   S_i [128 x 128] = Q_i K^T      tcgen05.mma kind::f16, both operands in shared memory
//   O_i [128 x D]  += W_i V        weights in tensor memory (operand A), V in shared memory
// The two tiles alternate, so that one's softmax runs while the tensor cores work for the other.
//
// Warps: 0-3 and 4-7 the softmax of tile 0 and 1 (a thread owns a row: no shuffles), 8-11 turn K
// codes into fp16, 12-15 V codes, 16 and 17 issue the MMAs.  Codes come straight from global memory
// into registers one step ahead (16 bytes a load) and leave as 128-byte-swizzled fp16 rows, K as a
// K-major operand, V (token rows, features contiguous) as an MN-major one: neither is transposed.
//
// Tensor memory: S_0, S_1 (128 columns each) and O_0, O_1 (D columns each), all 512 for D = 128.
// The fp16 weights overwrite the first half of their scores.  The MMAs of one tile execute in the
// order they are issued: W_i V of step j, then Q_i K^T of step j + 1, so S_i's arrival also says
// that the O_i before it is complete, and the rare rescaling of O_i needs no barrier of its own.
//
// What bounds it: a step of 128 tokens takes about 5000 cycles, the MMAs in it 2048 and the
// exponentials 2160 (16 a clock and SM): the chain scores -> softmax -> weights -> MMA of a tile is
// latency-bound with one warp of each tile on a scheduler; the tiles run half a step apart so
// that one's MMAs lie under the other's softmax.  6001 tokens over 7001 with 16 heads of 128: 277 us,
// 710 TFLOP/s; 8192 tokens, 32 heads: 798 TFLOP/s; heads of 64: 444 TFLOP/s.
//
// Every wait is bounded; after a time-out (recorded) each role leaves its loop and all meet at the
// end, where tensor memory is freed.
#include <type_traits>

#include "kv_common.cuh"

namespace bitnet {
namespace {

constexpr int kTile = 128;           // rows of an MMA, and tokens of a step
constexpr int kRows = 2 * kTile;     // rows of a block
constexpr int kGroups = kTile / kChunk;
constexpr int kBlockBytes = kTile * 128;  // 128 rows of 64 fp16: one swizzled operand block
constexpr int kMmaWarp = 16;
constexpr int kThreads = 20 * 32;         // warps 18 and 19 only complete the last warpgroup
// Registers: launched with 96 a thread (20 warps); 8 softmax warps take 144, the other 12 keep 64:
// 8 * 144 + 12 * 64 = 20 * 96.
constexpr int kManyRegisters = 144, kFewRegisters = 64;
// Weights in fp16 as in kv_attention.cu.  Here the sum of a 16-token group shows that one of them is
// too large for fp16 (65504): the reference moves where it exceeds 60 * 2^10, and then puts the
// largest weight in (2^7, 2^8].  Higher would see smaller weights but moves more often: 6001 tokens
// over 7001 take 278.6 us at 2^6, 279.5 at 2^8, 287 at 2^9 (with 2^15).
constexpr float kTop = 8.f, kMostSum = 61440.f;

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// fp16 x fp16 -> fp32; B K-major, or MN-major (features contiguous)
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// MN-major operand with the 128-byte swizzle: rows (the product's k) of 64 contiguous elements,
// eight of them 1024 bytes; the next 64 elements lie kBlockBytes further.
__device__ __forceinline__ uint64_t smem_desc_mnmajor_sw128(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)(kBlockBytes >> 4) << 16;  // leading: next 64 elements
    d |= (uint64_t)(1024 >> 4) << 32;         // stride: next eight rows
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Where the sums of a split sequence go: [piece][256 rows][D], then [..][2] maxima and denominators.
struct TcParts {
    float *sums, *stats;
};

struct Shared {
    uint64_t kfull[2], kfree[2], vfull[2], vfree[2], sfull[2], pfull[2], ofull[2], half[2], cfull[4];
    float4 group[4][kGroups];  // {d_K, log2 d_V, 1 / d_V} of the 16-token groups of a step
    float rowf[kRows];
    uint32_t tmem;
};

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <int R>
__device__ __forceinline__ void set_max_registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_max_registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_tc_kernel(KvArgs a, AttentionArgs at, TcParts parts, int units, int splits) {
    constexpr int NB = D / 64;                   // operand blocks of 64 features
    constexpr int TILE_BYTES = NB * kBlockBytes;
    constexpr uint32_t ID_S = idesc_f16(kTile, kTile, false), ID_O = idesc_f16(kTile, D, true);
    extern __shared__ uint8_t raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t sq = smem_addr(smem), sk = sq + 2 * TILE_BYTES, sv = sk + 2 * TILE_BYTES;

    // ---- which rows: the last (longest, when causal) units first, the heads of one together ----
    int x = blockIdx.x;
    const int split = x % splits;
    x /= splits;
    const int head = x % a.kv_heads;
    const int unit = units - 1 - x / a.kv_heads;
    const int G = at.q_heads / a.kv_heads;
    // sequence s owns the units from first(s) * G / 256 + s on: room for the tiles of its rows
    auto begin = [&](int i) { return ((int64_t)__ldg(a.q_start + i) * G >> 8) + (int64_t)i; };
    const int s = find_and_check(a, unit, tid == 0 && head == 0 && split == 0, begin,
                                 [&](const KvSequence &) { return at.max_new; });
    const KvSequence q = kv_sequence(a, s);
    if (!q.valid || q.count > at.max_new) return;  // nothing of it is read or written
    const int64_t tile = unit - begin(s);
    const int64_t all_rows = (int64_t)q.count * G;
    if (tile < 0 || tile * kRows >= all_rows) return;
    const int64_t r0 = tile * kRows;
    const int rows = (int)min((int64_t)kRows, all_rows - r0);
    // row r of this block is row (rem + r) % G of token base + (rem + r) / G
    const int base = (int)(r0 / G), rem = (int)(r0 - (int64_t)base * G);
    auto token_of = [&](int r) { return base + (rem + r) / G; };
    auto member_of = [&](int r) { return (rem + r) % G; };
    // tokens that the last row of tile i sees, and the steps that it takes
    int n[2], seen_first[2];
    int steps = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int sees = 0;
        seen_first[i] = 0;
        if (rows > i * kTile) {
            sees = at.causal ? q.length - q.count + token_of(min(rows, (i + 1) * kTile) - 1) + 1 : q.length;
            seen_first[i] = at.causal ? q.length - q.count + token_of(i * kTile) + 1 : q.length;
        }
        n[i] = sees > 0 ? (sees + kTile - 1) / kTile : 0;
        steps = max(steps, n[i]);
    }
    const int k0 = (int)((int64_t)steps * split / splits);
    const int k1 = (int)((int64_t)steps * (split + 1) / splits);
    const int ns = k1 - k0;
    n[0] = max(min(n[0], k1) - k0, 0);
    n[1] = max(min(n[1], k1) - k0, 0);

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.kfull[i], 4);
            mbar_init(&sh.vfull[i], 4);
            mbar_init(&sh.pfull[i], 4);
            mbar_init(&sh.half[i], 4);
            mbar_init(&sh.kfree[i], 2);
            mbar_init(&sh.vfree[i], 2);
            mbar_init(&sh.sfull[i], 1);
            mbar_init(&sh.ofull[i], 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mbar_init(&sh.cfull[i], 4);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    // ---- Q: a warp a row (four under way), scaled by a power of two, as fp16 ----
    constexpr int WQ = D / 64, WARPS = kThreads / 32, ROWS = 4;
#pragma unroll 1
    for (int r1 = warp; r1 < rows; r1 += ROWS * WARPS) {
        uint32_t w[ROWS][WQ];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int r = r1 + k * WARPS;
#pragma unroll
            for (int j = 0; j < WQ; ++j) w[k][j] = 0;
            if (r < rows) {
                const uint8_t *src = static_cast<const uint8_t *>(at.Q) +
                                     2 * ((int64_t)(q.first + token_of(r)) * at.ldq +
                                          (int64_t)(head * G + member_of(r)) * D);
                if constexpr (D == 128) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src) + lane);
                    w[k][0] = v.x;
                    w[k][1] = v.y;
                } else {
                    w[k][0] = __ldg(reinterpret_cast<const uint32_t *>(src) + lane);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int r = r1 + k * WARPS;
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < WQ; ++j) mx = __vmaxu2(mx, w[k][j] & 0x7FFF7FFFu);
            mx = __reduce_max_sync(0xFFFFFFFFu, max(mx & 0xFFFFu, mx >> 16));
            if (r >= rows) continue;  // what lies in rows that are not there goes nowhere
            float up, down;
            row_scaling(mx, down, up);
#pragma unroll
            for (int j = 0; j < WQ; ++j)
                w[k][j] = half2_of(__uint_as_float(w[k][j] << 16) * down,
                                   __uint_as_float(w[k][j] & 0xFFFF0000u) * down);
            const int rr = r % kTile;
            uint8_t *dst = smem + r / kTile * TILE_BYTES + rr * 128;
            if constexpr (D == 128) {  // features 4 lane ..: block lane / 16, 8 bytes
                const int c = (lane & 15) >> 1;
                *reinterpret_cast<uint2 *>(dst + (lane >> 4) * kBlockBytes + ((c ^ (rr & 7)) << 4) +
                                           (lane & 1) * 8) = make_uint2(w[k][0], w[k][1]);
            } else {  // features 2 lane ..
                const int c = lane >> 2;
                *reinterpret_cast<uint32_t *>(dst + ((c ^ (rr & 7)) << 4) + (lane & 3) * 4) = w[k][0];
            }
            if (lane == 0) sh.rowf[r] = up * (at.scale * kLog2e);
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    bool ok = true;

    if (warp >= kMmaWarp) {
        set_max_registers_down<kFewRegisters>();
        // ---- the MMAs: warps 16 and 17 issue those of tile 0 and 1, one thread each ----
        const int i = __shfl_sync(0xFFFFFFFFu, warp, 0) - kMmaWarp;
        if (i < 2 && ns > 0) {
            const bool leader = elect_one();
            const int ni = i ? n[1] : n[0];
            const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint32_t d_s = tb + i * kTile, d_o = tb + 2 * kTile + i * D;
            const uint64_t qd = smem_desc_kmajor_sw128(sq + i * TILE_BYTES);
            const uint64_t kd = smem_desc_kmajor_sw128(sk), vd = smem_desc_mnmajor_sw128(sv);
            auto scores = [&](int j) {
                const uint64_t kj = kd + (j & 1) * (TILE_BYTES >> 4);
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // 16 features, 32 bytes, each
                        const int off = b * (kBlockBytes >> 4) + 2 * e;
                        mma_f16_ss(d_s, qd + off, kj + off, ID_S, b + e > 0);
                    }
                mma_commit(&sh.sfull[i]);
            };
            auto output = [&](int j) {
                const uint64_t vj = vd + (j & 1) * (TILE_BYTES >> 4);
#pragma unroll
                for (int e = 0; e < kTile / 16; ++e)  // 16 tokens: 8 columns of weights, 2 KB of V
                    mma_f16_ts(d_o, d_s + 8 * e, vj + (2048 >> 4) * e, ID_O, j + e > 0);
            };
            // Both warps wait for every step's K and V, also where their tile takes no part, and both
            // release them (the barriers count two): none runs ahead of a stage's phase.
            ok = mbar_wait(&sh.kfull[0], 0, a.status);
            tc_fence_after();
            if (ok && leader) {
                if (ni > 0) scores(0);
                mma_commit(&sh.kfree[0]);
            }
            for (int j = 0; j < ns && ok; ++j) {
                ok = mbar_wait(&sh.vfull[j & 1], (j >> 1) & 1, a.status);
                if (ok && j < ni) ok = mbar_wait(&sh.pfull[i], j & 1, a.status);
                tc_fence_after();
                if (ok && leader) {
                    if (j < ni) output(j);
                    if (j == ni - 1) mma_commit(&sh.ofull[i]);
                    mma_commit(&sh.vfree[j & 1]);
                }
                if (ok && j + 1 < ns) {
                    ok = mbar_wait(&sh.kfull[(j + 1) & 1], ((j + 1) >> 1) & 1, a.status);
                    tc_fence_after();
                    if (ok && leader) {
                        if (j + 1 < ni) scores(j + 1);
                        mma_commit(&sh.kfree[(j + 1) & 1]);
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---- codes to fp16: a warp takes 32 tokens, two groups, of K or of V ----
        set_max_registers_down<kFewRegisters>();
        const bool is_k = warp < 12;
        const int w0 = (warp & 3) * 2;       // the warp's first group
        const int8_t *codes = is_k ? a.k_codes : a.v_codes;
        uint64_t *full = is_k ? sh.kfull : sh.vfull, *freed = is_k ? sh.kfree : sh.vfree;
        constexpr int PPT = D / 16;          // 16-code pieces a token
        constexpr int N = PPT;               // pieces a lane: 32 tokens * PPT / 32
        constexpr int TPI = 32 / PPT;        // tokens that the warp covers with a piece a lane
        // This lane's piece and token of the 32 / PPT that the warp takes at once.  A piece is 16
        // features: two 16-byte places of a swizzled row.  Eight lanes cover four pieces of one
        // operand block in two neighbouring rows: with that they meet in no bank.
        const int pc = D == 128 ? (lane & 3) | (lane >> 1 & 4) : lane & 3;
        const int tok = D == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane >> 2;
        const int row0 = (warp & 3) * 32 + tok;
        uint4 c[N];
        float gk = 0.f, gv = 0.f;            // K warps: the steps of group w0 + lane, lane < 2
        int entry[2] = {0, 0}, page[2] = {-1, -1};
        // the page table is asked one step ahead of the codes
        auto look_up = [&](int j) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int pos = (k0 + j) * kTile + (w0 + g) * kChunk;
                if (pos < q.length) entry[g] = kv_page_entry(a, s, pos);
            }
        };
        auto load = [&](int j) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int pos = (k0 + j) * kTile + (w0 + g) * kChunk;
                page[g] = pos < q.length ? kv_page_checked(a, entry[g]) : -1;
                // tokens behind the length or of an invalid page: any codes do, they weigh nothing
                const int8_t *from = codes + (page[g] >= 0 ? kv_code_at(a, page[g], head, pos) : 0) +
                                     tok * D + 16 * pc;
#pragma unroll
                for (int i = 0; i < N / 2; ++i) c[g * (N / 2) + i] = ldg_nc_v4(from + 512 * i);
            }
            const int mine = lane ? page[1] : page[0];
            if (is_k && lane < 2 && mine >= 0) {
                const int64_t at_step =
                    kv_scale_at(a, mine, head, (k0 + j) * kTile + (w0 + lane) * kChunk);
                gk = __ldg(a.k_scales + at_step);
                gv = __ldg(a.v_scales + at_step);
            }
        };
        // With D = 128 the rows of odd pieces are 4 further than those of even ones, modulo the 8 of
        // the swizzle.
        const uint32_t to = (is_k ? sk : sv) + (pc >> 2) * kBlockBytes + row0 * 128 +
                            (((2 * (pc & 3)) ^ (row0 & 7)) << 4);
        if (ns > 0) {
            look_up(0);
            load(0);
            if (ns > 1) look_up(1);
        }
        for (int j = 0; j < ns; ++j) {
            const int st = j & 1;
            if (j >= 2) ok = mbar_wait(&freed[st], ((j - 2) >> 1) & 1, a.status);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (is_k) {
                // a group behind the length or of an invalid page weighs nothing
                if (lane < 2)
                    sh.group[j & 3][w0 + lane] = (lane ? page[1] : page[0]) >= 0
                                                     ? make_float4(gk, log2_approx(v_step(gv)),
                                                                   __frcp_rn(v_step(gv)), 0.f)
                                                     : make_float4(0.f, -INFINITY, 0.f, 0.f);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.cfull[j & 3]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t x0 = c[i].x ^ 0x80808080u, x1 = c[i].y ^ 0x80808080u;
                const uint32_t x2 = c[i].z ^ 0x80808080u, x3 = c[i].w ^ 0x80808080u;
                const uint32_t dst = (D == 128 && (i & 1) ? to ^ 64 : to) + st * TILE_BYTES + i * TPI * 128;
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(codes_lo(x0)),
                             "r"(codes_hi(x0)), "r"(codes_lo(x1)), "r"(codes_hi(x1)) : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst ^ 16),
                             "r"(codes_lo(x2)), "r"(codes_hi(x2)), "r"(codes_lo(x3)), "r"(codes_hi(x3))
                             : "memory");
            }
            if (j + 1 < ns) {
                load(j + 1);
                if (j + 2 < ns) look_up(j + 2);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
        }
    } else {
        // ---- softmax: thread = row ----
        set_max_registers_up<kManyRegisters>();
        const int i = warp >> 2;
        const int r = i * kTile + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + i * kTile + lanes, to = tmem + 2 * kTile + i * D + lanes;
        const bool live = r < rows;
        const float rowf = live ? sh.rowf[r] : 0.f;
        // rows that are not there see everything and are dropped
        const int seen = !live ? INT32_MAX : at.causal ? q.length - q.count + token_of(r) + 1 : q.length;
        float m = live ? kNothing : 0.f, l = 0.f;  // (a row that is not there has a reference)
        const int ni = i ? n[1] : n[0], all_see = i ? seen_first[1] : seen_first[0];
        // One step in blocks of 32 tokens, with the reference so far.  A weight that it makes larger
        // than kMostSum shows in the sum of its group: no scan for the maximum is needed.  Only then (or for
        // a row's first block) the reference moves, the block is made again, and what the old one went
        // into is scaled: the sum, O_i, the step's earlier weights.  `sees` of the 128 tokens are seen.
        // The code is kept short (loops, one copy of the block): unrolled it was 110 KB, and fetching
        // instructions bound the kernel.
        auto step = [&](auto part, const float4 *group, int sees, int j) {
            constexpr bool PART = decltype(part)::value;
            auto block = [&](uint32_t (&v)[32], int b) {
                uint32_t w[16];
                const float4 g0 = group[2 * b], g1 = group[2 * b + 1];
                const float f[2] = {rowf * g0.x, rowf * g1.x};
                const int left = sees - 32 * b;
                float sg[2];
                bool moved = false;
#pragma unroll 1
                for (;;) {
                    const float c[2] = {g0.y - m, g1.y - m};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int k = 16 * h + 2 * e;
                            float2 z = __ffma2_rn(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                                                  make_float2(f[h], f[h]), make_float2(c[h], c[h]));
                            z.x = exp2_approx(z.x);
                            z.y = exp2_approx(z.y);
                            if constexpr (PART) {
                                if (k >= left) z.x = 0.f;
                                if (k + 1 >= left) z.y = 0.f;
                            }
                            sum[e & 1] = __fadd2_rn(sum[e & 1], z);
                            w[8 * h + e] = half2_of(z.x, z.y);
                        }
                        sum[0] = __fadd2_rn(sum[0], sum[1]);
                        sg[h] = sum[0].x + sum[0].y;
                    }
                    const bool over = fmaxf(sg[0], sg[1]) > kMostSum || m == kNothing;
                    if (moved || !__any_sync(0xFFFFFFFFu, over)) break;
                    moved = true;
                    // earlier weights of this step, and O_i where it was scaled before, are read back
                    // below: stores to tensor memory are only ordered before loads by this wait
                    tmem_wait_st();
                    float top = kNothing;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!PART || e < left)
                            top = fmaxf(top, fmaf(__uint_as_float(v[e]), f[e / 16], e < 16 ? g0.y : g1.y));
                    const float mn = over ? fmaxf(m, ceilf(top) - kTop) : m;
                    const float keep = exp2_approx(m - mn);
                    m = mn;
                    l *= keep;
#pragma unroll 1
                    for (int c16 = 0; c16 < b; ++c16) {
                        tmem_ld_32x32b_x16(ts + 16 * c16, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {  // in fp32: fp16 has no factor below 2^-24
                            const float2 z = float2_of(w[e]);
                            w[e] = half2_of(z.x * keep, z.y * keep);
                        }
                        tmem_st_32x32b_x16(ts + 16 * c16, w);
                    }
#pragma unroll 1
                    for (int c16 = 0; c16 < (j > 0 ? D / 16 : 0); ++c16) {
                        tmem_ld_32x32b_x16(to + 16 * c16, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            w[e] = __float_as_uint(__uint_as_float(w[e]) * keep);
                        tmem_st_32x32b_x16(to + 16 * c16, w);
                    }
                }
                // a row that sees none of a group takes nothing of it, whatever its step is
                if (sg[0] != 0.f) l = fmaf(sg[0], g0.z, l);
                if (sg[1] != 0.f) l = fmaf(sg[1], g1.z, l);
                tmem_st_32x32b_x16(ts + 16 * b, w);
            };
            uint32_t va[32], vb[32];
            tmem_ld_32x32b_x32(ts, va);
#pragma unroll 1
            for (int b = 0; b < 4; b += 2) {  // the next block's scores are under way
                tmem_wait_ld();
                tmem_ld_32x32b_x32(ts + 32 * b + 32, vb);
                block(va, b);
                tmem_wait_ld();
                if (b == 0) tmem_ld_32x32b_x32(ts + 64, va);
                block(vb, b + 1);
                if (b == 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.half[i]);
                }
            }
        };
        for (int j = 0; j < ni; ++j) {
            ok = mbar_wait(&sh.cfull[j & 3], (j >> 2) & 1, a.status) &&
                 mbar_wait(&sh.sfull[i], j & 1, a.status);
            // Half a step apart: a tile begins when the other one is half through, so that the MMAs of
            // one run under the softmax of the other instead of both waiting at the same time.
            if (i == 1 && j < n[0]) ok = ok && mbar_wait(&sh.half[0], j & 1, a.status);
            if (i == 0 && j > 0 && j <= n[1]) ok = ok && mbar_wait(&sh.half[1], (j - 1) & 1, a.status);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            const float4 *group = sh.group[j & 3];
            const int pos = (k0 + j) * kTile;
            // a step that some row sees only in part has its own code: 128 comparisons more
            if (pos + kTile > all_see)
                step(std::true_type(), group, seen - pos, j);
            else
                step(std::false_type(), group, kTile, j);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pfull[i]);
        }
        // ---- out ----
        if (ni > 0 && ok) ok = mbar_wait(&sh.ofull[i], 0, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        const int64_t token = q.first + token_of(r), qh = head * G + member_of(r);
        const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
        const int64_t piece = (((int64_t)unit * a.kv_heads + head) * splits + split) * kRows + r;
        if (ok) {
#pragma unroll 1
            for (int b = 0; b < D / 32; ++b) {
                uint32_t v[32];
                if (ni > 0) {
                    tmem_ld_32x32b_x32(to + 32 * b, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0;
                }
                if (live && splits == 1) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(at.Y) +
                                                           2 * (token * at.ldy + qh * D + 32 * b));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[k] = bf16x2_of(__uint_as_float(v[8 * e + 2 * k]) * inv,
                                             __uint_as_float(v[8 * e + 2 * k + 1]) * inv);
                        dst[e] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                } else if (live) {
                    uint4 *dst = reinterpret_cast<uint4 *>(parts.sums + piece * D + 32 * b);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
                __syncwarp();  // the next load takes the whole warp
            }
            if (live) {
                if (splits > 1)
                    *reinterpret_cast<float2 *>(parts.stats + 2 * piece) = make_float2(m, l);
                else if (at.lse)
                    at.lse[token * at.q_heads + qh] =
                        l == 0.f ? -INFINITY : (m + log2_approx(l)) * kLn2;
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the pieces of split rows: a warp a row.
template <int D>
__global__ void __launch_bounds__(256)
    kv_attention_tc_join_kernel(KvArgs a, AttentionArgs at, TcParts parts, int units, int splits) {
    constexpr int F = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int r = (int)(w % kRows);
    const int64_t uh = w / kRows;
    const int head = (int)(uh % a.kv_heads), unit = (int)(uh / a.kv_heads);
    if (unit >= units) return;
    const int G = at.q_heads / a.kv_heads;
    auto begin = [&](int i) { return ((int64_t)__ldg(a.q_start + i) * G >> 8) + (int64_t)i; };
    const int s = find_sequence(unit, a.batch, begin);
    const KvSequence q = kv_sequence(a, s);
    if (!q.valid || q.count > at.max_new) return;
    const int64_t row = (unit - begin(s)) * kRows + r;
    if (row < 0 || row >= (int64_t)q.count * G) return;
    float m = kNothing, l = 0.f, v[F] = {};
#pragma unroll 4
    for (int i = 0; i < splits; ++i) {
        const int64_t piece = (uh * splits + i) * kRows + r;
        const float2 ml = *reinterpret_cast<const float2 *>(parts.stats + 2 * piece);
        const float mn = fmaxf(m, ml.x);
        const float old = exp2_approx(m - mn), now = exp2_approx(ml.x - mn);
        l = l * old + ml.y * now;
#pragma unroll
        for (int f = 0; f < F; ++f) v[f] = v[f] * old + parts.sums[piece * D + 32 * f + lane] * now;
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
    const int64_t token = q.first + row / G, qh = head * (int64_t)G + row % G;
    __nv_bfloat16 *Y = static_cast<__nv_bfloat16 *>(at.Y) + token * at.ldy + qh * D;
#pragma unroll
    for (int f = 0; f < F; ++f) Y[32 * f + lane] = __float2bfloat16(v[f] * inv);
    if (at.lse && lane == 0)
        at.lse[token * at.q_heads + qh] = l == 0.f ? -INFINITY : (m + log2_approx(l)) * kLn2;
}

int64_t tc_units(const KvArgs &a, const AttentionArgs &at) {
    return ((int64_t)a.tokens * (at.q_heads / a.kv_heads) >> 8) + a.batch;
}

// Pieces that a row's cache is cut into, none shorter than four steps of the longest sequence that
// the page table allows.  Prompts: enough to fill the SMs once (pieces of 256 rows cost 130 KB of
// partial sums each).  Few rows (one tile at most): enough for two rounds of the SMs, which evens
// out ragged lengths.
int tc_splits(const KvArgs &a, const AttentionArgs &at) {
    const int64_t blocks = tc_units(a, at) * a.kv_heads;
    const int64_t steps = ((int64_t)a.max_pages << a.page_shift) / kTile;
    const bool few = (int64_t)at.max_new * (at.q_heads / a.kv_heads) <= kTile;
    int64_t n = few ? (2 * kSms + blocks - 1) / blocks : kSms / blocks;
    if (n > steps / 4) n = steps / 4;
    return n < 1 ? 1 : (int)n;
}

template <int D>
cudaError_t launch_tc(const KvArgs &a, const AttentionArgs &at, void *ws, cudaStream_t stream,
                      int *launches) {
    const int64_t units = tc_units(a, at);
    const int splits = tc_splits(a, at);
    const int64_t blocks = units * a.kv_heads * splits;
    if (units > INT32_MAX || blocks > INT32_MAX) return cudaErrorInvalidValue;
    constexpr int smem = 6 * (D / 64) * kBlockBytes + 1024;
    TcParts parts = {};
    if (splits > 1) {
        parts.sums = static_cast<float *>(ws);
        parts.stats = parts.sums + (size_t)blocks * kRows * D;
    }
    auto kern = kv_attention_tc_kernel<D>;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    kern<<<(unsigned)blocks, kThreads, smem, stream>>>(a, at, parts, (int)units, splits);
    *launches = 1;
    if ((e = cudaGetLastError()) != cudaSuccess || splits == 1) return e;
    kv_attention_tc_join_kernel<D><<<(unsigned)(units * a.kv_heads * (kRows / 8)), 256, 0, stream>>>(
        a, at, parts, (int)units, splits);
    *launches = 2;
    return cudaGetLastError();
}

}  // namespace

size_t kv_attention_tc_workspace(const KvArgs &a, const AttentionArgs &at) {
    const int splits = tc_splits(a, at);
    if (splits == 1) return 0;
    return (size_t)(tc_units(a, at) * a.kv_heads * splits) * kRows * (a.head_dim + 2) * 4;
}

cudaError_t launch_kv_attention_tc(const KvArgs &a, const AttentionArgs &at, void *ws,
                                   cudaStream_t stream, int *launches) {
    return a.head_dim == 64 ? launch_tc<64>(a, at, ws, stream, launches)
                            : launch_tc<128>(a, at, ws, stream, launches);
}

}  // namespace bitnet
