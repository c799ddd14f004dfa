"""GPU parity of the residual norm quantiser, the paged 8-bit K/V cache and attention over it.

References: tests/kv_reference.py (codes and steps bit for bit, attention in 64 bits with the error
bound derived there), the CPU oracle for the activation codes.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import oracle
from bit_activation_linear_b200 import synth

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0**-8   # half a step of bf16, relative


@pytest.fixture(scope="module")
def B():
    from bit_activation_linear_b200 import build, binding
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load_library()
    return binding


def bf16(a):
    """float32 values -> (bf16 torch tensor on the GPU, the float32 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16()
    return t.cuda(), t.float().numpy()


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def to_device(B, cache):
    return B.KvCache(*(torch.from_numpy(a.copy()).cuda() for a in cache.codes),
                     *(torch.from_numpy(a.copy()).cuda() for a in cache.steps))


class Batch:
    """Sequences of given lengths with their last `new` tokens, pages in random order."""

    def __init__(self, lengths, new, page, rng, spare=2, gap=0, behind=0):
        self.kv_len, self.new = list(lengths), list(new)
        self.q_start = [gap]
        for n in new:
            self.q_start.append(self.q_start[-1] + n)
        self.tokens = self.q_start[-1] + behind
        count = [-(-n // page) for n in self.kv_len]
        self.pages = sum(count) + spare
        order = list(rng.permutation(self.pages))
        width = max(max(count), 1) + 1
        self.table = np.full((len(count), width), -7, np.int32)   # entries behind the length
        for s, c in enumerate(count):
            self.table[s, :c] = [order.pop() for _ in range(c)]

    def device(self):
        return ints(self.q_start), ints(self.kv_len), ints(self.table)


def same_cache(got, want):
    for a, b in zip((got.k_codes, got.v_codes), want.codes):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    for a, b in zip((got.k_scales, got.v_scales), want.steps):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


# ----------------------------------------------------------------------------------------
# residual addition + RMS norm + codes
# ----------------------------------------------------------------------------------------

RES_SHAPES = [(1, 128), (3, 384), (1, 2048), (130, 2048), (5, 4096), (37, 5120), (2, 8192),
              (3, 32768), (2, 33024), (1, 65536)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K", RES_SHAPES)
def test_residual_norm_matches_the_separate_steps(B, M, K, bits):
    """H bit for bit; the codes against 64 bits.  A code may differ by one where its value lies
    within e of a tie: rinv carries the fp32 sum of K squares (any order: K / 2 partial sums of at
    most log2 K + 32 levels, bounded by 64 half steps), three roundings of its own, and y * s three
    more, so e = 2 * 70 * 2^-24 * |value| <= 127 * 140 * 2^-24 < 1.1e-3."""
    rng = np.random.default_rng(K + M + bits)
    X, x = bf16(rng.standard_normal((M, K)) * 0.3)
    r = rng.standard_normal((M, K)).astype(np.float32)
    r[:, :: max(1, K // 7)] *= 20
    R, r = bf16(r)
    G, g = bf16(1 + 0.2 * rng.standard_normal(K))
    for gain, gv in ((G, g), (None, np.ones(K, np.float32))):
        H, codes, scales, rowsum = B.bitnet_act_quant_residual_norm(X, R, gain, 1e-5, bits)
        B.bitnet_sync_status()
        want_h = (torch.from_numpy(x) + torch.from_numpy(r)).bfloat16()
        assert torch.equal(H.cpu(), want_h)
        h = want_h.double().numpy()
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5) * gv.astype(np.float64)
        if bits == 8:
            top = np.maximum(np.abs(y).max(1), 1e-5)
            pre, step = y * (127 / top)[:, None], top / 127
        else:
            mean = np.maximum(np.abs(y).mean(1), 1e-5)
            pre = np.clip(y * (7 ** 0.5 / mean)[:, None], -8, 7)
            step = mean / 7 ** 0.5
        got = codes.cpu().numpy()
        if bits == 4:
            w = got.view(np.uint8).reshape(M, K // 8, 4)
            nib = np.concatenate([w & 15, w >> 4], 2).reshape(M, K).astype(np.int16)
            got = np.where(nib > 7, nib - 16, nib)
        got = got.astype(np.int64)
        diff = got - np.rint(pre).astype(np.int64)
        off = diff != 0
        assert np.abs(diff).max() <= 1
        assert np.all(np.abs(np.abs(pre[off] - np.floor(pre[off])) - 0.5) < 1.1e-3)
        np.testing.assert_allclose(scales.cpu().numpy(), step, rtol=140 * 2.0**-24)
        np.testing.assert_array_equal(rowsum.cpu().numpy(), got.sum(1))


def test_residual_norm_in_place_and_equal_to_the_norm_of_the_sum(B):
    rng = np.random.default_rng(3)
    X, _ = bf16(rng.standard_normal((66, 2048)))
    R, _ = bf16(rng.standard_normal((66, 2048)) * 3)
    H, codes, scales, rowsum = B.bitnet_act_quant_residual_norm(X, R, None, 1e-6, 8)
    ref_codes, ref_scales, ref_sum = B.bitnet_act_quant_norm(H, None, 1e-6, False, 8)
    # the two kernels sum the squares in different orders: codes within 1.1e-3 of a tie (the bound
    # of the test above) may differ, by one
    diff = (codes.int() - ref_codes.int()).abs()
    assert diff.max() <= 1 and diff.sum() <= 2.2e-3 * diff.numel()
    for target in ("X", "R"):
        x, r = X.clone(), R.clone()
        out = {"X": x, "R": r}[target]
        h2, c2, s2, m2 = B.bitnet_act_quant_residual_norm(x, r, None, 1e-6, 8, H=out)
        assert h2.data_ptr() == out.data_ptr()
        assert torch.equal(h2, H) and torch.equal(c2, codes)
        assert torch.equal(s2, scales) and torch.equal(m2, rowsum)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M", [1, 33, 200])
def test_residual_norm_forward_is_the_quantiser_and_the_product(B, M, bits):
    rng = np.random.default_rng(M)
    K, N = 1024, 256
    X, _ = bf16(rng.standard_normal((M, K)))
    R, _ = bf16(rng.standard_normal((M, K)))
    G, _ = bf16(1 + 0.1 * rng.standard_normal(K))
    W = synth.to_torch_bf16(synth.latent_weights(N, K, seed=5)).cuda()
    Wp, gamma = B.bitnet_quantize_pack_weights(W)
    H, Y = B.bitnet_residual_norm_bitlinear_forward(X, R, G, 1e-5, Wp, gamma, bits)
    h, codes, scales, rowsum = B.bitnet_act_quant_residual_norm(X, R, G, 1e-5, bits)
    _, y = B.bitnet_ternary_gemm(codes, scales, rowsum, K, Wp, gamma, bits)
    B.bitnet_sync_status()
    assert torch.equal(H, h) and torch.equal(Y, y)


def test_residual_norm_zero_and_nonfinite_rows_stay_apart(B):
    X = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    R = torch.zeros_like(X)
    R[1] = 1.0
    R[2, 7] = float("nan")
    R[3] = -2.0
    H, codes, scales, rowsum = B.bitnet_act_quant_residual_norm(X, R, None, 1e-5, 8)
    B.bitnet_sync_status()
    assert codes[0].eq(0).all() and rowsum[0] == 0
    assert codes[1].eq(127).all() and codes[3].eq(-127).all()
    assert torch.isnan(H[2, 7]) and rowsum[3] == -127 * 512


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("K", [128, 2048, 33024])
def test_residual_norm_nonfinite_rows_show(B, bits, K):
    """A row with a NaN or an infinity gets codes of 0 and a scale that is NaN, so whatever is made of
    it is NaN; the rows beside it (of the same block for small K) are what they are without it."""
    rng = np.random.default_rng(K)
    X, _ = bf16(rng.standard_normal((9, K)))
    R, _ = bf16(rng.standard_normal((9, K)))
    clean = B.bitnet_act_quant_residual_norm(X, R, None, 1e-5, bits)
    X[1, K - 1] = float("nan")
    R[3, 0] = float("inf")
    X[4] = float("-inf")
    X[6, 5], R[6, 5] = float("inf"), float("-inf")
    bad = [1, 3, 4, 6]
    good = [i for i in range(9) if i not in bad]
    H, codes, scales, rowsum = B.bitnet_act_quant_residual_norm(X, R, None, 1e-5, bits)
    B.bitnet_sync_status()
    assert torch.equal(H.isnan() | H.isinf(), ~(X.float() + R.float()).isfinite())
    assert torch.isnan(scales[bad]).all() and torch.all(codes[bad] == 0)
    assert torch.all(rowsum[bad] == 0)
    for got, want in zip((H, codes, scales, rowsum), clean):
        assert torch.equal(got[good], want[good])
    # a gain that is infinite where the row is not zero
    G = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    G[7] = float("inf")
    X, R = (t.clone() for t in (X, R))
    X[0], R[0] = 0.0, 0.0                  # 0 * inf
    X[2], R[2] = 1.0, 1.0
    _, codes, scales, _ = B.bitnet_act_quant_residual_norm(X, R, G, 1e-5, bits)
    assert torch.isnan(scales[0]) and torch.isinf(scales[2])
    assert torch.all(codes[[0, 2]] == 0)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M", [1, 6, 40, 300])
def test_residual_norm_forward_of_nonfinite_rows_is_nan(B, bits, M):
    """On every product kernel the output row of a NaN or infinite row is NaN, and no other."""
    rng = np.random.default_rng(M)
    K, N = 1024, 256
    X, _ = bf16(rng.standard_normal((M, K)))
    R, _ = bf16(rng.standard_normal((M, K)))
    W = synth.to_torch_bf16(synth.latent_weights(N, K, seed=5)).cuda()
    Wp, gamma = B.bitnet_quantize_pack_weights(W)
    _, clean = B.bitnet_residual_norm_bitlinear_forward(X, R, None, 1e-5, Wp, gamma, bits)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    for row, value in ((0, "nan"), (M // 2, "inf"), (M - 1, "-inf")):
        X[row, row] = float(value)
        bad[row] = True
    H, Y = B.bitnet_residual_norm_bitlinear_forward(X, R, None, 1e-5, Wp, gamma, bits)
    B.bitnet_sync_status()
    assert torch.isnan(Y[bad]).all()
    assert torch.equal(Y[~bad], clean[~bad])


# ----------------------------------------------------------------------------------------
# cache: append and read back
# ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (32, 16), (64, 64), (256, 32), (128, 128)])
@pytest.mark.parametrize("heads", [1, 5])
def test_append_bit_exact_over_several_calls(B, dim, page, block, heads):
    """Prompts, single tokens and chunks that end inside blocks and pages, one call after the
    other; lengths of 0 and 1 among them; rows before and behind the sequences are not read."""
    rng = np.random.default_rng(dim + page + heads)
    final = [0, 1, page, page + 1, 3 * page - 1, 2 * block + 5]
    layout = Batch(final, [0] * 6, page, rng)
    cache = ref.Cache(layout.pages, heads, dim, page, block, rng)
    got = to_device(B, cache)
    length = [0] * len(final)
    scale = 1.0
    while length != final:
        new = [min(f - n, int(rng.choice([0, 1, 2, 7, block, page + 3])))
               for f, n in zip(final, length)]
        length = [n + k for n, k in zip(length, new)]
        step = Batch(length, new, page, rng, gap=2, behind=3)
        scale *= float(rng.choice([0.3, 1.0, 2.5]))   # later tokens that are larger
        shape = (step.tokens, heads, dim)
        K, k = bf16(rng.standard_normal(shape) * scale)
        V, v = bf16(rng.standard_normal(shape) * rng.uniform(0.01, 3, (1, heads, 1)))
        K[:2] = float("nan")
        V[step.q_start[-1]:] = float("inf")
        cache.append((k, v), step.q_start, length, layout.table)
        B.bitnet_kv_cache_append(got, K, V, ints(step.q_start), ints(length),
                                 ints(layout.table))
    B.bitnet_sync_status()
    same_cache(got, cache)


def test_append_of_strided_slices_and_large_ratios(B):
    """Column slices of a wider product; steps that grow by 2^20 and by one unit in the last
    place; zero states."""
    rng = np.random.default_rng(8)
    heads, dim, page, block = 2, 64, 32, 16
    layout = Batch([9], [9], page, rng)
    cache = ref.Cache(layout.pages, heads, dim, page, block, rng)
    got = to_device(B, cache)
    wide = np.zeros((9, 5 * heads * dim), np.float32)
    mags = [0.0, 1e-7, 1.0, 1.0, 1.0078125, 2.0**20, 3.0, 3e38, 1.0]
    for t, m in enumerate(mags):
        wide[t] = rng.uniform(-m, m, wide.shape[1])
        wide[t, ::heads * dim // 2] = m
    W, w = bf16(wide)
    width = heads * dim
    for t in range(9):
        K, V = W[t:t + 1, width:2 * width], W[t:t + 1, 3 * width:4 * width]
        k, v = w[t:t + 1, width:2 * width], w[t:t + 1, 3 * width:4 * width]
        cache.append([a.reshape(1, heads, dim) for a in (k, v)], [0, 1], [t + 1], layout.table)
        B.bitnet_kv_cache_append(got, K, V, ints([0, 1]), ints([t + 1]), ints(layout.table))
    same_cache(got, cache)
    # all nine at once, rows apart
    cache = ref.Cache(layout.pages, heads, dim, page, block, rng)
    got = to_device(B, cache)
    cache.append([w[:, width:2 * width].reshape(9, heads, dim),
                  w[:, 3 * width:4 * width].reshape(9, heads, dim)], [0, 9], [9], layout.table)
    B.bitnet_kv_cache_append(got, W[:, width:2 * width], W[:, 3 * width:4 * width],
                             ints([0, 9]), ints([9]), ints(layout.table))
    B.bitnet_sync_status()
    same_cache(got, cache)


def test_append_nonfinite_states_mark_their_block_only(B):
    rng = np.random.default_rng(9)
    heads, dim, page = 2, 64, 32
    layout = Batch([40], [40], page, rng)
    cache = ref.Cache(layout.pages, heads, dim, page, 16, rng)
    clean = to_device(B, cache)
    dirty = to_device(B, cache)
    K, _ = bf16(rng.standard_normal((40, heads, dim)))
    V, _ = bf16(rng.standard_normal((40, heads, dim)))
    K2, V2 = K.clone(), V.clone()
    K2[20, 1, 5] = float("nan")
    V2[3, 0, 9] = float("-inf")
    meta = [ints([0, 40]), ints([40]), ints(layout.table)]
    B.bitnet_kv_cache_append(clean, K, V, *meta)
    B.bitnet_kv_cache_append(dirty, K2, V2, *meta)
    B.bitnet_sync_status()
    p0, p1 = int(layout.table[0, 0]), int(layout.table[0, 1])
    assert torch.isnan(dirty.k_scales[p0, 1, 1]) and torch.isinf(dirty.v_scales[p0, 0, 0])
    dirty.k_scales[p0, 1, 1] = clean.k_scales[p0, 1, 1]
    dirty.v_scales[p0, 0, 0] = clean.v_scales[p0, 0, 0]
    assert torch.equal(dirty.k_scales, clean.k_scales)
    assert torch.equal(dirty.v_scales, clean.v_scales)
    # a further token in a NaN block does not hide it; one that begins the block anew does
    B.bitnet_kv_cache_append(dirty, K2[:40], V2[:40], *meta)
    B.bitnet_kv_cache_append(dirty, K[:2], V[:2], ints([0, 2]), ints([32]), meta[2])
    assert torch.isnan(dirty.k_scales[p0, 1, 1])
    B.bitnet_kv_cache_append(dirty, K, V, *meta)
    assert torch.isfinite(dirty.k_scales[p0]).all() and torch.isfinite(dirty.v_scales[p1]).all()
    B.bitnet_sync_status()


@pytest.mark.parametrize("dim,page,block", [(64, 16, 16), (128, 64, 16), (128, 256, 256)])
def test_read_back(B, dim, page, block):
    rng = np.random.default_rng(dim + page)
    heads = 3
    lengths = [1, 0, 2 * page + 9, 77, page]
    new = [1, 0, 2 * page + 9, 20, 5]
    b = Batch(lengths, new, page, rng, gap=1, behind=2)
    cache = ref.Cache(b.pages, heads, dim, page, block, rng)
    got = to_device(B, cache)
    width = heads * dim
    outs = [torch.full((b.tokens, width + 8), 7.0, dtype=torch.bfloat16, device="cuda")
            for _ in range(2)]
    K, V = B.bitnet_kv_cache_read(got, b.tokens, *b.device(), K=outs[0][:, :width],
                                  V=outs[1][:, 8:])
    B.bitnet_sync_status()
    for which, (out, lo) in enumerate(((outs[0], 0), (outs[1], 8))):
        want = np.full((b.tokens, width + 8), 7.0, np.float32)
        for s, length in enumerate(lengths):
            if new[s]:
                c, d = cache.states(which, s, length, b.table)
                v = (c.astype(np.float32) * d.astype(np.float32)[..., None])[:, length - new[s]:]
                want[b.q_start[s]:b.q_start[s + 1], lo:lo + width] = v.transpose(1, 0, 2).reshape(
                    new[s], width)
        assert torch.equal(out.cpu(), torch.from_numpy(want).bfloat16())
    same_cache(got, cache)


# ----------------------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------------------

def filled(B, rng, lengths, new, heads, dim, page, block, k_scale=1.0, **more):
    """A cache that holds the batch's states (unused places keep what they held)."""
    b = Batch(lengths, new, page, rng, **more)
    cache = ref.Cache(b.pages, heads, dim, page, block, rng)
    total = sum(lengths)
    k = rng.standard_normal((total, heads, dim)).astype(np.float32) * k_scale
    k[:, :, ::29] *= 5
    v = rng.standard_normal((total, heads, dim)).astype(np.float32)
    v *= rng.uniform(0.2, 4, (total, heads, 1)).astype(np.float32)
    starts = [0] + list(np.cumsum(lengths))
    cache.append((bf16(k)[1], bf16(v)[1]), starts, lengths, b.table)
    return b, cache, to_device(B, cache)


def check_attention(B, b, cache, got, q_heads, causal=True, scale=None, max_new=None, **more):
    rng = np.random.default_rng(q_heads)
    dim = cache.codes[0].shape[3]
    Q, q = bf16(rng.standard_normal((b.tokens, q_heads * dim)))
    Y = torch.full((b.tokens, q_heads * dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.tokens, q_heads), 7.0, device="cuda")
    B.bitnet_kv_attention(got, Q, q_heads, *b.device(), max_new or max(max(b.new), 1),
                          scale=scale, causal=causal, Y=Y, lse=lse, **more)
    B.bitnet_sync_status()
    scale = dim ** -0.5 if scale is None else scale
    y, l, tol_y, tol_l = ref.attention(cache, q.astype(np.float64).reshape(-1, q_heads, dim),
                                       b.q_start, b.kv_len, b.table, scale, causal)
    a, z = b.q_start[0], b.q_start[-1]
    Yn = Y.float().cpu().numpy().reshape(-1, q_heads, dim)
    ln = lse.cpu().numpy()
    assert np.all(Yn[:a] == 7) and np.all(Yn[z:] == 7), "rows of no sequence were written"
    assert np.all(ln[:a] == 7) and np.all(ln[z:] == 7)
    Yn, ln, y, l = Yn[a:z], ln[a:z], y[a:z], l[a:z]
    err = np.abs(Yn - y) - (BF16_HALF * np.abs(y) + tol_y[a:z] * (1 + BF16_HALF))
    assert err.max(initial=-1) <= 0, err.max()
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(ln), empty) and np.all(Yn[empty] == 0)
    assert np.all(np.abs(ln[~empty] - l[~empty]) <= tol_l[a:z][~empty])
    return Y, lse


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 4, 8, 12, 16, 17, 32, 33])
def test_attention_single_tokens_ragged(B, dim, group):
    rng = np.random.default_rng(dim + group)
    lengths = [1, 15, 16, 17, 300, 64, 129]
    b, cache, got = filled(B, rng, lengths, [1] * 7, 2, dim, 64, 16, gap=1, behind=2)
    check_attention(B, b, cache, got, 2 * group)


@pytest.mark.parametrize("page,block", [(16, 16), (32, 32), (64, 16), (128, 64), (256, 256)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new", [1, 3, 6])
def test_attention_a_few_tokens_pages_and_blocks(B, page, block, causal, new):
    rng = np.random.default_rng(page + block + new)
    lengths = [new, page, 2 * page + 1, page - 1 + new, 513]
    b, cache, got = filled(B, rng, lengths, [new, 1, new, min(new, 2), new], 3, 128, page, block)
    check_attention(B, b, cache, got, 9, causal=causal)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,lengths", [
    ([17], [17]), ([33, 64], [33, 200]), ([129], [129]), ([128, 1, 40], [640, 77, 41]),
    ([300], [333]), ([257, 0, 100], [300, 50, 100])])
@pytest.mark.parametrize("group", [1, 4, 7])
def test_attention_prompts(B, dim, new, lengths, group):
    rng = np.random.default_rng(sum(new) + group + dim)
    b, cache, got = filled(B, rng, lengths, new, 2, dim, 32, 16, gap=1, behind=3)
    check_attention(B, b, cache, got, 2 * group)


@pytest.mark.parametrize("new", [1, 5, 60])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_rows_that_see_nothing(B, new, causal):
    """Lengths of 0, and fewer tokens than new ones: the first rows see nothing when causal."""
    rng = np.random.default_rng(new)
    b, cache, got = filled(B, rng, [0, 3, 0, max(new - 2, 0), 20], [new, new, 0, new, new], 2, 64,
                           16, 16, behind=1)
    check_attention(B, b, cache, got, 8, causal=causal)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_garbage_behind_the_length_is_not_seen(B, new):
    """NaN and infinite steps of blocks that are not seen: behind the length, and in pages of
    nobody."""
    rng = np.random.default_rng(new)
    b, cache, got = filled(B, rng, [new + 70, 45], [new, min(new, 45)], 2, 128, 64, 16)
    want = check_attention(B, b, cache, got, 8)
    used = np.zeros((b.pages, 4), bool)
    for s, length in enumerate(b.kv_len):
        for t in range(0, length, 16):
            used[b.table[s, t // 64], t % 64 // 16] = True
    hole = torch.from_numpy(~used).cuda()[:, None, :].expand_as(got.k_scales)
    got.k_scales[hole] = float("nan")
    got.v_scales[hole] = float("inf")
    again = check_attention(B, b, cache, got, 8)
    assert all(torch.equal(x, y) for x, y in zip(want, again))


@pytest.mark.parametrize("new", [1, 40])
def test_attention_nonfinite_values_reach_their_rows_only(B, new):
    rng = np.random.default_rng(new + 1)
    b, cache, got = filled(B, rng, [200, 100], [new, new], 2, 128, 64, 16)
    dim, q_heads = 128, 8
    Q, _ = bf16(rng.standard_normal((b.tokens, q_heads * dim)))
    meta = b.device()
    Y0, l0 = B.bitnet_kv_attention(got, Q, q_heads, *meta, new, want_lse=True)
    Q2 = Q.clone()
    Q2[0, 3 * dim + 7] = float("nan")      # row 0, head 3
    Q2[-1, 6 * dim] = float("inf")         # last row, head 6
    Y1, l1 = B.bitnet_kv_attention(got, Q2, q_heads, *meta, new, want_lse=True)
    bad = torch.zeros((b.tokens, q_heads), dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[-1, 6] = True
    per = Y1.view(-1, q_heads, dim)
    assert torch.isnan(per[bad]).all() and torch.isnan(l1[bad]).all()
    assert torch.equal(per[~bad], Y0.view(-1, q_heads, dim)[~bad])
    assert torch.equal(l1[~bad], l0[~bad])
    # a block with a NaN or infinite step: the rows of its head that see it, and no others
    for steps, value in ((got.k_scales, "nan"), (got.k_scales, "inf"), (got.v_scales, "nan")):
        keep = steps.clone()
        steps[int(b.table[1, 0]), 1, 2] = float(value)     # sequence 1, head 1, positions 32-47
        got.k_codes[int(b.table[1, 0]), 1, 32:48] = 0
        Y2, _ = B.bitnet_kv_attention(got, Q, q_heads, *meta, new)
        first = b.kv_len[1] - new
        rows = [b.q_start[1] + i for i in range(new) if first + i >= 32]
        per = Y2.view(-1, q_heads, dim)
        assert torch.isnan(per[rows, 4:]).all()
        assert torch.equal(per[:b.q_start[1]], Y0.view(-1, q_heads, dim)[:b.q_start[1]])
        assert torch.equal(per[:, :4], Y0.view(-1, q_heads, dim)[:, :4])
        steps.copy_(keep)
    B.bitnet_sync_status()


@pytest.mark.parametrize("bits", [0xFFFFFFFF, 0x7FFFFFFF, 0x7FC00000, 0xFFC00000, 0x7F800001])
@pytest.mark.parametrize("new", [1, 9, 40])
def test_attention_shows_any_nan_step(B, new, bits):
    """Whatever the NaN's bits: the rows of its head that see the block are NaN, and no others."""
    rng = np.random.default_rng(2)
    heads, dim = 2, 64
    b, cache, got = filled(B, rng, [200], [new], heads, dim, 64, 16)
    Q, _ = bf16(rng.standard_normal((new, 2 * heads * dim)))
    clean, _ = B.bitnet_kv_attention(got, Q, 2 * heads, *b.device(), new)
    for steps in (got.k_scales, got.v_scales):
        keep = steps.clone()
        steps.view(torch.int32)[int(b.table[0, 0]), 1, 2] = bits - 2**32 if bits >= 2**31 else bits
        Y, lse = B.bitnet_kv_attention(got, Q, 2 * heads, *b.device(), new, want_lse=True)
        B.bitnet_sync_status()
        assert torch.isnan(Y[:, 2 * dim:]).all() and torch.isnan(lse[:, 2:]).all()
        assert torch.equal(Y[:, :2 * dim], clean[:, :2 * dim])
        steps.copy_(keep)


@pytest.mark.parametrize("q_scale,k_scale", [(1e-20, 1e10), (1e20, 1e-20), (300.0, 1.0),
                                             (1e-3, 1e-6)])
@pytest.mark.parametrize("new", [1, 30])
def test_attention_large_and_small_magnitudes(B, q_scale, k_scale, new):
    rng = np.random.default_rng(4)
    b, cache, got = filled(B, rng, [333, 50], [new, new], 1, 64, 32, 32, k_scale=k_scale)
    # V steps that differ by ten decimal orders between blocks
    factor = 10.0 ** rng.uniform(-5, 5, cache.steps[1].shape)
    cache.steps[1] = (cache.steps[1] * factor).astype(np.float32)
    got = to_device(B, cache)
    rng = np.random.default_rng(5)
    Q, q = bf16(rng.standard_normal((b.tokens, 4 * 64)) * q_scale)
    Y, lse = B.bitnet_kv_attention(got, Q, 4, *b.device(), new, want_lse=True)
    B.bitnet_sync_status()
    y, l, tol_y, tol_l = ref.attention(cache, q.astype(np.float64).reshape(-1, 4, 64), b.q_start,
                                       b.kv_len, b.table, 0.125, True)
    got_y = Y.float().cpu().numpy().reshape(y.shape)
    assert np.all(np.abs(got_y - y) <= BF16_HALF * np.abs(y) + tol_y * (1 + BF16_HALF))
    assert np.all(np.abs(lse.cpu().numpy() - l) <= tol_l)


@pytest.mark.parametrize("batch,length,new", [(1, 5000, 1), (3, 2500, 2), (2, 3000, 20)])
def test_attention_long_axis_is_split_and_joined(B, batch, length, new):
    rng = np.random.default_rng(length)
    b, cache, got = filled(B, rng, [length - 13 * i for i in range(batch)], [new] * batch, 2, 64,
                           64, 16)
    first = check_attention(B, b, cache, got, 8)
    again = check_attention(B, b, cache, got, 8)
    assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_attention_strided_rows_and_hints(B):
    """Q as a column slice of a fused product, Y inside a wider buffer; a max_new that is larger
    than any sequence needs gives the same up to the kernels' rounding."""
    rng = np.random.default_rng(6)
    heads, dim, q_heads = 2, 64, 6
    b, cache, got = filled(B, rng, [50, 90], [1, 1], heads, dim, 32, 16)
    qkv, q = bf16(rng.standard_normal((2, (q_heads + 2 * heads) * dim)))
    out = torch.full((2, q_heads * dim + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    y, l, tol_y, _ = ref.attention(
        cache, q[:, :q_heads * dim].astype(np.float64).reshape(2, q_heads, dim), b.q_start,
        b.kv_len, b.table, 0.2, True)
    for hint in (1, 2, 9, 1000):
        out.fill_(7.0)
        B.bitnet_kv_attention(got, qkv[:, :q_heads * dim], q_heads, *b.device(), hint, scale=0.2,
                              Y=out[:, 8:8 + q_heads * dim])
        B.bitnet_sync_status()
        o = out.float().cpu().numpy()
        assert np.all(o[:, :8] == 7) and np.all(o[:, 8 + q_heads * dim:] == 7)
        o = o[:, 8:8 + q_heads * dim].reshape(y.shape)
        assert np.all(np.abs(o - y) <= BF16_HALF * np.abs(y) + tol_y * (1 + BF16_HALF))


@pytest.mark.parametrize("new", [1, 40])
def test_sequences_that_share_pages(B, new):
    """A common prefix in pages that two sequences read gives what copies of the pages give."""
    rng = np.random.default_rng(new)
    heads, dim, page = 2, 64, 32
    cache = B.KvCache.empty(12, heads, dim, page, 16)
    table = ints([[3, 7, 1, 2], [5, 6, 0, 4]])
    prefix = bf16(rng.standard_normal((64, heads * dim)))[0]
    tails = bf16(rng.standard_normal((2 * new, heads * dim)))[0]
    twice = torch.cat([prefix, prefix])
    B.bitnet_kv_cache_append(cache, twice, twice, ints([0, 64, 128]), ints([64, 64]), table)
    meta = ints([0, new, 2 * new]), ints([64 + new, 64 + new])
    B.bitnet_kv_cache_append(cache, tails, tails, *meta, table)
    Q = bf16(rng.standard_normal((2 * new, 4 * dim)))[0]
    want = B.bitnet_kv_attention(cache, Q, 4, *meta, table, new, want_lse=True)
    shared = ints([[3, 7, 1, 2], [3, 7, 0, 4]])
    got = B.bitnet_kv_attention(cache, Q, 4, *meta, shared, new, want_lse=True)
    B.bitnet_sync_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_beyond_32_bits(B):
    """Pages whose codes lie more than 2^31 and 2^32 bytes into the cache give what the same pages
    give in a small one: writing, reading back and both attention kernels."""
    rng = np.random.default_rng(17)
    heads, dim, page, block, q_heads = 2, 128, 256, 16, 4
    tile = heads * page * dim
    places = [3, 2**31 // tile + 1, 2**32 // tile + 2]          # positions 0.., 256.., 512..
    pages = places[-1] + 2
    big = B.KvCache.empty(pages, heads, dim, page, block)
    small = B.KvCache.empty(4, heads, dim, page, block)
    length = 600
    states = [bf16(rng.standard_normal((length, heads * dim)))[0] for _ in range(2)]
    tables = {big: ints([places]), small: ints([[2, 0, 3]])}
    results = []
    for cache in (big, small):
        table = tables[cache]
        B.bitnet_kv_cache_append(cache, states[0][:599], states[1][:599], ints([0, 599]),
                                 ints([599]), table)
        B.bitnet_kv_cache_append(cache, states[0][599:], states[1][599:], ints([0, 1]),
                                 ints([600]), table)
        out = list(B.bitnet_kv_cache_read(cache, 600, ints([0, 600]), ints([600]), table))
        for new in (1, 50):
            Q = torch.from_numpy(np.random.default_rng(new).standard_normal(
                (new, q_heads * dim)).astype(np.float32)).bfloat16().cuda()
            out += B.bitnet_kv_attention(cache, Q, q_heads, ints([0, new]), ints([600]), table, new,
                                         want_lse=True)
        results.append(out)
    B.bitnet_sync_status()
    assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("batch", [130, 1100])
def test_many_sequences(B, batch):
    """More sequences than a block has threads, most of them short or empty, in every call."""
    rng = np.random.default_rng(batch)
    heads, dim, page = 1, 64, 16
    lengths = [int(x) for x in rng.integers(0, 40, batch)]
    new = [min(n, int(rng.integers(0, 3))) for n in lengths]
    b, cache, got = filled(B, rng, lengths, new, heads, dim, page, 16, gap=1, behind=2)
    check_attention(B, b, cache, got, 2, max_new=2)
    check_attention(B, b, cache, got, 2, max_new=40)
    shape = (b.tokens, heads, dim)
    K, k = bf16(rng.standard_normal(shape) * 3)
    V, v = bf16(rng.standard_normal(shape) * 3)
    cache.append((k, v), b.q_start, b.kv_len, b.table)
    B.bitnet_kv_cache_append(got, K, V, *b.device())
    B.bitnet_sync_status()
    same_cache(got, cache)


def test_attention_scores_that_keep_growing_and_falling(B):
    """The maximum moves in every chunk, or never again after the first one: rising and falling
    keys, by steps below and above what moves it, for both kernels."""
    for new in (1, 40):
        for slope in (0.9, -0.9, 0.05, -0.05):
            rng = np.random.default_rng(3)
            heads, dim, page, length = 1, 64, 32, 700
            b = Batch([length], [new], page, rng)
            cache = ref.Cache(b.pages, heads, dim, page, 16, rng)
            k = rng.standard_normal((length, heads, dim)).astype(np.float32) * 0.1
            k[:, 0, 0] = slope * np.arange(length)
            v = rng.standard_normal((length, heads, dim)).astype(np.float32)
            cache.append((bf16(k)[1], bf16(v)[1]), [0, length], [length], b.table)
            got = to_device(B, cache)
            Q, q = bf16(np.abs(rng.standard_normal((b.tokens, 2 * dim))) + 0.5)
            Y, lse = B.bitnet_kv_attention(got, Q, 2, *b.device(), new, want_lse=True)
            B.bitnet_sync_status()
            y, l, tol_y, tol_l = ref.attention(cache, q.astype(np.float64).reshape(-1, 2, dim),
                                               b.q_start, b.kv_len, b.table, dim ** -0.5, True)
            got_y = Y.float().cpu().numpy().reshape(y.shape)
            assert np.all(np.abs(got_y - y) <= BF16_HALF * np.abs(y) + tol_y * (1 + BF16_HALF))
            assert np.all(np.abs(lse.cpu().numpy() - l) <= tol_l)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("jump", [9, 13])
@pytest.mark.parametrize("run", [16, 32, 48])
def test_attention_maxima_that_move_several_times_in_a_step(B, dim, jump, run):
    """Scores that rise by 2^jump every `run` tokens: the prompt kernel scales the weights it has
    already stored for a step of 128 tokens, and the sums of earlier steps, up to eight times in that
    step.  The highest tokens have zero V codes in half of the features, whose outputs are then made
    of what was scaled."""
    heads, page, block = 2, 64, 16
    lengths, new = [130, 200, 333, 460], [40, 33, 60, 35]
    rng = np.random.default_rng(jump + run)
    b = Batch(lengths, new, page, rng)
    cache = ref.Cache(b.pages, heads, dim, page, block, rng)
    for s, length in enumerate(lengths):
        for t in range(length):
            at = (b.table[s, t // page], slice(None), t % page)
            cache.codes[0][at] = 0
            level = t // run
            cache.codes[0][at + (0,)] = 4 * level        # times a step of jump / 4, in powers of two
            cache.codes[1][at] = rng.integers(60, 120, (heads, dim))
            if level == (length - 1) // run:
                cache.codes[1][at][:, : dim // 2] = 0
    cache.steps[0][:] = jump / 4
    cache.steps[1][:] = 0.01
    got = to_device(B, cache)
    q = np.zeros((b.tokens, heads, dim), np.float32)
    q[:, :, 0] = 1
    Q, q = bf16(q)
    scale = float(np.float32(np.log(2.0)))
    Y, lse = B.bitnet_kv_attention(got, Q.flatten(1), heads, *b.device(), max(new), scale=scale,
                                   want_lse=True)
    B.bitnet_sync_status()
    y, l, tol_y, tol_l = ref.attention(cache, q.astype(np.float64), b.q_start, b.kv_len, b.table,
                                       scale, True)
    got_y = Y.float().cpu().numpy().reshape(y.shape)
    assert np.all(np.abs(got_y - y) <= BF16_HALF * np.abs(y) + tol_y * (1 + BF16_HALF))
    assert np.all(np.abs(lse.cpu().numpy() - l) <= tol_l)


# ----------------------------------------------------------------------------------------
# what the device finds wrong; streams and graphs
# ----------------------------------------------------------------------------------------

def test_invalid_sequences_and_pages_are_reported_and_left_out(B):
    rng = np.random.default_rng(12)
    heads, dim, page = 2, 64, 16
    b, cache, got = filled(B, rng, [40, 33, 20], [2, 2, 2], heads, dim, page, 16)
    K, k = bf16(rng.standard_normal((6, heads * dim)))
    Q, q = bf16(rng.standard_normal((6, 4 * dim)))
    start, length, table = b.device()

    def status(call):
        call()
        with pytest.raises(B.BitnetError) as e:
            B.bitnet_sync_status()
        assert e.value.status == B.ERR_INVALID
        B.bitnet_sync_status()   # cleared

    cases = [
        (ints([0, 2, 900, 6]), length, table),            # rows outside the matrix
        (ints([0, 2, -1, 6]), length, table),             # rows that go back
        (start, ints([40, 100000, 20]), table),           # longer than its page table
        (start, ints([40, -1, 20]), table),
    ]
    for meta in cases:
        before = [t.clone() for t in (got.k_codes, got.v_codes, got.k_scales, got.v_scales)]
        Y = torch.full((6, 4 * dim), 7.0, dtype=torch.bfloat16, device="cuda")
        out = torch.full((6, heads * dim), 7.0, dtype=torch.bfloat16, device="cuda")
        status(lambda: B.bitnet_kv_attention(got, Q, 4, *meta, 2, Y=Y))
        status(lambda: B.bitnet_kv_cache_read(got, 6, *meta, K=out, V=out.clone()))
        assert torch.all(Y[2:4] == 7) and torch.all(out[2:4] == 7)
        status(lambda: B.bitnet_kv_cache_append(got, K, K, *meta))
        for t, was in zip((got.k_codes, got.v_codes, got.k_scales, got.v_scales), before):
            t.copy_(was)
    # more new tokens than max_new says
    status(lambda: B.bitnet_kv_attention(got, Q, 4, start, length, table, 1))
    # pages that are not there: their tokens are not seen, everything else is
    for wrong in (-1, b.pages, 2**31 - 1):
        bad = b.table.copy()
        bad[1, 0] = wrong
        Y = torch.full((6, 4 * dim), 7.0, dtype=torch.bfloat16, device="cuda")
        status(lambda: B.bitnet_kv_attention(got, Q, 4, start, length, ints(bad), 2, Y=Y))
        good = B.bitnet_kv_attention(got, Q, 4, start, length, table, 2)[0]
        assert torch.equal(Y[:2], good[:2]) and torch.equal(Y[4:], good[4:])
        assert torch.isfinite(Y[2:4].float()).all()
        bad[1, :] = wrong
        out = torch.full((6, heads * dim), 7.0, dtype=torch.bfloat16, device="cuda")
        status(lambda: B.bitnet_kv_cache_read(got, 6, start, length, ints(bad), K=out,
                                              V=out.clone()))
        assert torch.all(out[2:4] == 7) and not torch.any(out[:2] == 7)
        status(lambda: B.bitnet_kv_cache_append(got, K, K, start, length, ints(bad)))
    B.bitnet_kv_cache_append(got, K, K, start, length, table)
    B.bitnet_sync_status()


def reported(B, call):
    call()
    with pytest.raises(B.BitnetError) as e:
        B.bitnet_sync_status()
    assert e.value.status == B.ERR_INVALID
    B.bitnet_sync_status()   # cleared


@pytest.mark.parametrize("q_start,tokens", [
    ([0, 900, 3, 6], 6), ([43, 187, 0, 237], 400), ([141, 313, 205, 288], 400),
    ([0, 200, 400, 0, 0, 10], 400), ([-5, 4, 8], 8), ([0, 4, 9], 8), ([0] * 40 + [300] + [7] * 30, 9),
    (list(range(50)) + [20] + list(range(51, 70)), 70)])
def test_q_start_that_goes_back_is_reported(B, q_start, tokens):
    """Whichever blocks find the sequence: by every call, and rows that no valid sequence claims stay
    as they were."""
    heads, dim, page, group = 1, 64, 64, 4
    n = len(q_start) - 1
    cache = B.KvCache.empty(8 * n + 1, heads, dim, page, 16)
    for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
        t.zero_()
    table = ints(np.arange(8 * n).reshape(n, 8))
    meta = ints(q_start), ints([512] * n), table
    claimed = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    for lo, hi in zip(q_start, q_start[1:]):
        if 0 <= lo <= hi <= tokens:
            claimed[lo:hi] = True
    K = torch.ones((tokens, heads * dim), dtype=torch.bfloat16, device="cuda")
    reported(B, lambda: B.bitnet_kv_cache_append(cache, K, K, *meta))
    assert not cache.k_codes[8 * n].any() and not cache.v_scales[8 * n].any()
    out = [torch.full_like(K, 7.0) for _ in range(2)]
    reported(B, lambda: B.bitnet_kv_cache_read(cache, tokens, *meta, K=out[0], V=out[1]))
    for t in out:
        assert torch.all(t[~claimed] == 7)
    Q = torch.ones((tokens, group * dim), dtype=torch.bfloat16, device="cuda")
    for max_new in (8, 400):          # streaming (longer sequences are invalid there), prompts
        Y = torch.full_like(Q, 7.0)
        lse = torch.full((tokens, group), 7.0, device="cuda")
        reported(B, lambda: B.bitnet_kv_attention(cache, Q, group, *meta, max_new, Y=Y, lse=lse))
        assert torch.all(Y[~claimed] == 7) and torch.all(lse[~claimed] == 7)


@pytest.mark.parametrize("new,group", [(2, 4), (8, 4), (20, 4), (70, 8)])
def test_invalid_sequences_and_pages_of_both_attention_kernels(B, new, group):
    rng = np.random.default_rng(new)
    heads, dim, page = 2, 64, 16
    b, cache, got = filled(B, rng, [new + 40, new + 33, new + 20], [new] * 3, heads, dim, page, 16)
    q_heads = heads * group
    Q, q = bf16(rng.standard_normal((b.tokens, q_heads * dim)))
    start, length, table = b.device()
    good, good_lse = B.bitnet_kv_attention(got, Q, q_heads, start, length, table, new, want_lse=True)

    def call(*meta, **more):
        Y = torch.full((b.tokens, q_heads * dim), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b.tokens, q_heads), 7.0, device="cuda")
        reported(B, lambda: B.bitnet_kv_attention(got, Q, q_heads, *meta, new, Y=Y, lse=lse, **more))
        return Y, lse

    mid = slice(new, 2 * new)
    for bad in (-1, 100000, 2**31 - 1):
        Y, lse = call(start, ints([b.kv_len[0], bad, b.kv_len[2]]), table)
        assert torch.all(Y[mid] == 7) and torch.all(lse[mid] == 7)
        for rows in (slice(0, new), slice(2 * new, None)):
            assert torch.equal(Y[rows], good[rows]) and torch.equal(lse[rows], good_lse[rows])
    # a page that is not there: as if its tokens were not in the sequence
    short = [b.kv_len[0], b.kv_len[1] - page, b.kv_len[2]]
    without = b.table.copy()
    without[1, :-1] = b.table[1, 1:]
    y, l, tol_y, tol_l = ref.attention(cache, q.astype(np.float64).reshape(-1, q_heads, dim),
                                       b.q_start, short, without, dim ** -0.5, False)
    for wrong in (-1, b.pages, 2**31 - 1):
        bad = b.table.copy()
        bad[1, 0] = wrong
        Y, lse = call(start, length, ints(bad), causal=False)
        got_y = Y.float().cpu().numpy().reshape(y.shape)
        assert np.all(np.abs(got_y - y) <= BF16_HALF * np.abs(y) + tol_y * (1 + BF16_HALF))
        assert np.all(np.abs(lse.cpu().numpy() - l) <= tol_l)
        # a sequence without any page sees nothing
        bad[1, :] = wrong
        Y, lse = call(start, length, ints(bad))
        assert torch.all(Y[mid] == 0) and torch.all(lse[mid] == -float("inf"))
        assert torch.equal(Y[:new], good[:new]) and torch.equal(Y[2 * new:], good[2 * new:])


def test_empty_calls_do_nothing(B):
    rng = np.random.default_rng(1)
    b, cache, got = filled(B, rng, [5], [1], 1, 64, 16, 16)
    none = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    meta = (ints([0, 0]), ints([5]), ints(b.table))
    B.bitnet_kv_cache_append(got, none, none, *meta)
    K, V = B.bitnet_kv_cache_read(got, 0, *meta)
    Y, lse = B.bitnet_kv_attention(got, none, 1, *meta, 1, want_lse=True)
    assert K.shape == V.shape == Y.shape == (0, 64) and lse.shape == (0, 1)
    nobody = (ints([0]), ints([]), torch.empty((0, 3), dtype=torch.int32, device="cuda"))
    some = torch.full((2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    B.bitnet_kv_attention(got, some.clone(), 1, *nobody, 1, Y=some)
    B.bitnet_sync_status()
    assert torch.all(some == 7)
    same_cache(got, cache)


@pytest.mark.parametrize("max_new", [1, 9, 300])
def test_empty_batches_of_either_kernel_do_nothing(B, max_new):
    """A scheduler with nobody to serve: the call allocates its own workspace."""
    rng = np.random.default_rng(1)
    b, cache, got = filled(B, rng, [5], [1], 4, 64, 16, 16)
    nobody = (ints([0]), ints([]), torch.empty((0, 3), dtype=torch.int32, device="cuda"))
    for tokens in (0, 2):
        Q = torch.full((tokens, 16 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
        Y = Q.clone()
        assert B.bitnet_kv_attention_workspace_bytes(got, tokens, 0, 3, 16, max_new) == 0
        B.bitnet_kv_attention(got, Q, 16, *nobody, max_new, Y=Y)
        assert torch.equal(Y, Q)
    none = torch.empty((0, 16 * 64), dtype=torch.bfloat16, device="cuda")
    B.bitnet_kv_attention(got, none, 16, ints([0, 0]), ints([5]), ints(b.table), max_new)
    B.bitnet_sync_status()
    same_cache(got, cache)


@pytest.mark.parametrize("new", [1, 24])
def test_attention_on_two_streams_and_in_replayed_graphs(B, new):
    """Two calls at once with a workspace each; a graph replayed with other lengths, pages and
    queries in the same buffers."""
    rng = np.random.default_rng(21)
    b, cache, got = filled(B, rng, [3000, 100], [new, new], 2, 64, 64, 16)
    Q, _ = bf16(rng.standard_normal((b.tokens, 8 * 64)))
    start, length, table = b.device()
    want = B.bitnet_kv_attention(got, Q, 8, start, length, table, new, want_lse=True)
    shorter = ints([1234, 100])
    want2 = B.bitnet_kv_attention(got, Q, 8, start, shorter, table, new, want_lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(20):
        for s, lens in zip(streams, (length, shorter)):
            outs.append(B.bitnet_kv_attention(got, Q, 8, start, lens, table, new, want_lse=True,
                                              stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        w = (want, want2)[i % 2]
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    lens = length.clone()
    Y = torch.empty_like(want[0])
    lse = torch.empty_like(want[1])
    ws = torch.empty(max(16, B.bitnet_kv_attention_workspace_bytes(
        got, b.tokens, 2, table.shape[1], 8, new)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.bitnet_kv_attention(got, Q, 8, start, lens, table, new, Y=Y, lse=lse, ws=ws)
    for value, w in ((shorter, want2), (length, want), (shorter, want2)):
        lens.copy_(value)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, w[0]) and torch.equal(lse, w[1])
    B.bitnet_sync_status()


def test_calls_from_several_host_threads(B):
    """A thread a stream, each with its own cache: writes, reads back and attention of both kernels and
    head sizes at once give what they give one after the other."""
    import threading

    def work(dim, seed, stream, out):
        with torch.cuda.stream(stream):
            gen = torch.Generator(device="cuda").manual_seed(seed)

            def rand(*shape):
                return torch.randn(shape, generator=gen, device="cuda").bfloat16()

            cache = B.KvCache.empty(20, 2, dim)
            table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
            meta = ints([0, 700]), ints([700]), table
            B.bitnet_kv_cache_append(cache, rand(700, 2 * dim), rand(700, 2 * dim), *meta)
            out += B.bitnet_kv_cache_read(cache, 700, *meta)
            for new, heads in ((1, 4), (5, 8), (80, 4)):
                for _ in range(10):
                    out += B.bitnet_kv_attention(cache, rand(new, heads * dim), heads, ints([0, new]),
                                                 ints([700]), table, new, want_lse=True)
            stream.synchronize()

    jobs = [(dim, seed, torch.cuda.Stream()) for dim in (64, 128) for seed in range(4)]
    want = []
    for job in jobs:
        want.append([])
        work(*job, want[-1])
    got = [[] for _ in jobs]
    threads = [threading.Thread(target=work, args=(*job, out)) for job, out in zip(jobs, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
    B.bitnet_sync_status()


@pytest.mark.parametrize("own_stream", [False, True])
def test_chains_of_calls_that_nothing_waits_between(B, own_stream):
    """Writes and attention of growing sequences, one call after the other, give what they give with
    a synchronisation behind every call (the kernels are launched before the ones they follow end)."""
    heads, dim, group = 2, 128, 4
    stream = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()
    results = []
    with torch.cuda.stream(stream):
        table = torch.arange(80, dtype=torch.int32, device="cuda").view(4, 20)
        for wait in (False, True):
            cache = B.KvCache.empty(80, heads, dim)
            gen = torch.Generator(device="cuda").manual_seed(1)
            rng = np.random.default_rng(2)
            length, out = np.zeros(4, int), []
            for step in range(40):
                new = rng.integers(0, 4 if step % 10 else 60, 4)
                length = length + new
                if not new.sum():
                    continue
                meta = ints(np.concatenate([[0], np.cumsum(new)])), ints(length), table
                qkv = torch.randn((int(new.sum()), (group + 2) * heads * dim), generator=gen,
                                  device="cuda").bfloat16()
                q, k, v = qkv.split([group * heads * dim, heads * dim, heads * dim], 1)
                B.bitnet_kv_cache_append(cache, k, v, *meta)
                out += B.bitnet_kv_attention(cache, q, group * heads, *meta, int(new.max()),
                                             want_lse=True)
                if wait:
                    torch.cuda.synchronize()
            B.bitnet_sync_status()
            results.append(out)
    assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("M", [8, 32, 64])
def test_attention_right_behind_the_product_that_makes_its_queries(B, M):
    """Products and attention on the same buffers in turn, in a replayed graph and with nothing
    between them: the attention is launched while the product still runs, and reads its queries."""
    heads, dim, group = 2, 64, 4
    rng = np.random.default_rng(M)
    b, cache, got = filled(B, rng, [400, 100], [M // 2, M // 2], heads, dim, 64, 16)
    meta = b.device()
    width, K = heads * group * dim, 2048
    W = synth.to_torch_bf16(synth.latent_weights(width, K, seed=3)).cuda()
    Wp, gamma = B.bitnet_quantize_pack_weights(W)
    X = torch.stack([bf16(rng.standard_normal((M, K)))[0] for _ in range(8)])
    want = []
    for x in X:
        Q = B.bitnet_bitlinear_forward(x, Wp, gamma, 8)
        torch.cuda.synchronize()
        want.append(B.bitnet_kv_attention(got, Q, heads * group, *meta, M // 2, want_lse=True))
        torch.cuda.synchronize()
    Q = torch.empty((M, width), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.bitnet_workspace_bytes(M, K, width, 8), dtype=torch.uint8, device="cuda")
    B.bitnet_bitlinear_forward(X[0], Wp, gamma, 8, Y=Q, ws=ws)
    outs = []

    def chain():
        outs.clear()
        for x in X:
            B.bitnet_bitlinear_forward(x, Wp, gamma, 8, Y=Q, ws=ws)
            outs.append(B.bitnet_kv_attention(got, Q, heads * group, *meta, M // 2, want_lse=True))

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(20):
        for o in outs:
            o[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    B.bitnet_sync_status()


def test_a_layer_step_residual_norm_qkv_cache_attention(B):
    """The operators one after the other as a decoder layer runs them: residual norm and Q/K/V
    product, cache write, attention, H-BitLinear output projection; a prompt, then single tokens,
    checked against the same chain in 64 bits from the operators' own stored codes."""
    rng = np.random.default_rng(30)
    width, q_heads, heads, dim, page = 256, 4, 2, 64, 32
    n_qkv = (q_heads + 2 * heads) * dim
    Wqkv, g1 = B.bitnet_quantize_pack_weights(
        synth.to_torch_bf16(synth.latent_weights(n_qkv, width, seed=1)).cuda())
    Wo, g2 = B.bitnet_quantize_pack_weights(
        synth.to_torch_bf16(synth.latent_weights(width, q_heads * dim, seed=2)).cuda())
    G, _ = bf16(1 + 0.1 * rng.standard_normal(width))
    cache = B.KvCache.empty(8, heads, dim, page, 16)
    table = ints([[5, 2, 0], [1, 7, 4]])
    host = ref.Cache(8, heads, dim, page, 16, rng)
    length = [0, 0]
    for new in ([30, 41], [1, 1], [1, 1], [3, 2]):
        length = [a + n for a, n in zip(length, new)]
        start = [0, new[0], sum(new)]
        X, _ = bf16(rng.standard_normal((sum(new), width)))
        R, _ = bf16(rng.standard_normal((sum(new), width)))
        H, qkv = B.bitnet_residual_norm_bitlinear_forward(X, R, G, 1e-5, Wqkv, g1, 8)
        Q = qkv[:, :q_heads * dim]
        K = qkv[:, q_heads * dim:(q_heads + heads) * dim]
        V = qkv[:, (q_heads + heads) * dim:]
        B.bitnet_kv_cache_append(cache, K, V, ints(start), ints(length), table)
        Y, lse = B.bitnet_kv_attention(cache, Q, q_heads, ints(start), ints(length), table,
                                       max(new), want_lse=True)
        out = B.bitnet_hbitlinear_forward(Y, Wo, g2, 8)
        B.bitnet_sync_status()
        assert torch.isfinite(out.float()).all() and out.shape == X.shape
        host.append([t.float().cpu().numpy().reshape(-1, heads, dim) for t in (K, V)], start,
                    length, table.cpu().numpy())
        y, l, tol_y, tol_l = ref.attention(
            host, Q.double().cpu().numpy().reshape(-1, q_heads, dim), start, length,
            table.cpu().numpy(), dim ** -0.5, True)
        got = Y.double().cpu().numpy().reshape(y.shape)
        assert np.all(np.abs(got - y) <= BF16_HALF * np.abs(y) + tol_y * (1 + BF16_HALF))
        assert np.all(np.abs(lse.cpu().numpy() - l) <= tol_l)
        back = B.bitnet_kv_cache_read(cache, sum(length), ints([0, length[0], sum(length)]),
                                      ints(length), table)
        for which in (0, 1):
            rows = []
            for s in (0, 1):
                c, d = host.states(which, s, length[s], table.cpu().numpy())
                rows.append((c * d[..., None]).transpose(1, 0, 2).reshape(length[s], -1))
            want = np.concatenate(rows)
            assert np.all(np.abs(back[which].double().cpu().numpy() - want)
                          <= BF16_HALF * np.abs(want))


@pytest.mark.parametrize("batch", [1, 4, 12])
@pytest.mark.parametrize("bits", [8, 4])
def test_a_replayed_decoding_step(B, batch, bits):
    """Two layers of a decoder step captured once and replayed for 40 tokens, on one workspace and with
    lengths that grow on the device, give what the same calls give one by one."""
    width, q_heads, heads, dim, page = 512, 8, 2, 64, 16
    n_qkv = (q_heads + 2 * heads) * dim
    layers = []
    for i in (1, 2):
        layers.append([B.bitnet_quantize_pack_weights(
            synth.to_torch_bf16(synth.latent_weights(n, k, seed=10 * i)).cuda())
            for n, k in ((n_qkv, width), (width, q_heads * dim))])
    table = torch.randperm(4 * batch, generator=torch.Generator().manual_seed(1)).int().cuda()
    table = table.view(batch, 4)
    gen = torch.Generator(device="cuda").manual_seed(2)
    first = torch.randn((batch, width), generator=gen, device="cuda").bfloat16()
    start = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    need = max(B.bitnet_workspace_bytes(batch, k, n, bits) for n, k in ((n_qkv, width),
                                                                        (width, q_heads * dim)))

    class State:
        def __init__(self):
            self.caches = [B.KvCache.empty(4 * batch, heads, dim, page, 16) for _ in layers]
            for c in self.caches:
                for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
                    t.zero_()
            self.length = torch.arange(batch, dtype=torch.int32, device="cuda")
            self.stream, self.x = first.clone(), torch.zeros_like(first)
            self.qkv = torch.empty((batch, n_qkv), dtype=torch.bfloat16, device="cuda")
            self.y = torch.empty((batch, q_heads * dim), dtype=torch.bfloat16, device="cuda")
            self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def step(self, wait=lambda: None):
            self.length += 1
            for cache, (qkv_w, out_w) in zip(self.caches, layers):
                wait()
                B.bitnet_residual_norm_bitlinear_forward(self.x, self.stream, None, 1e-5, *qkv_w, bits,
                                                         H=self.stream, Y=self.qkv, ws=self.ws)
                q, k, v = self.qkv.split([q_heads * dim, heads * dim, heads * dim], 1)
                wait()
                B.bitnet_kv_cache_append(cache, k, v, start, self.length, table)
                wait()
                B.bitnet_kv_attention(cache, q, q_heads, start, self.length, table, 1, Y=self.y)
                wait()
                B.bitnet_hbitlinear_forward(self.y, *out_w, bits, Y=self.x, ws=self.ws)
                wait()

    one, other = State(), State()
    other.step()                       # first calls outside the capture
    other = State()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.step()
    for _ in range(40):
        one.step(torch.cuda.synchronize)
        graph.replay()
    torch.cuda.synchronize()
    B.bitnet_sync_status()
    assert torch.isfinite(one.stream.float()).all()
    for a, b in ((one.stream, other.stream), (one.x, other.x), (one.length, other.length)):
        assert torch.equal(a, b)
    for c, d in zip(one.caches, other.caches):
        assert torch.equal(c.k_codes, d.k_codes) and torch.equal(c.v_codes, d.v_codes)
        assert torch.equal(c.k_scales, d.k_scales) and torch.equal(c.v_scales, d.v_scales)
