"""What the attention kernels' fp16 weights and queries may lose: scores that jump, tokens that hold
nearly all of a row's weight, query features of very different size.

One sequence (or many that share its pages) whose codes and steps are made by hand: the key's first
feature is the score in powers of two, and V codes that are small where the weight is large show what
becomes of the small weights.  Expected values in 64 bits.

The bound, in units of code * step (D features, `seen` tokens, p the softmax weights):
* a score: D * 2^-22 * sum |q c| d scale, and 2^-21 * (1 + |s|) for exp2 (see kv_reference.py);
* a weight p d_V is rounded to 11 bits, 2^-11 of it, or to a fixed point, 2^-25 units.  The row's
  largest is above 2^6 units when the reference moves last and only rises, so that is 2^-31 of it.  In
  the prompt kernel it is above 2^7, 2^-32; a stored weight that is scaled (by a power of two below
  2^-1) is rounded once more for each move, which at most doubles it: 2^-31 covers both;
* sums of `seen` terms in fp32: seen * 2^-24; the output: half a step of bf16.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

LN2 = float(np.float32(np.log(2.0)))
PAGE, BLOCK = 64, 16


@pytest.fixture(scope="module")
def B():
    from bit_activation_linear_b200 import build, binding
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load_library()
    return binding


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def make_cache(B, k, v, dk, dv):
    """k, v int8 [tokens, dim]; dk, dv float [tokens / BLOCK]: a cache of one head, pages in order."""
    pages, dim = k.shape[0] // PAGE, k.shape[1]

    def steps(d):
        d = np.ascontiguousarray(d, np.float32).reshape(pages, 1, PAGE // BLOCK)
        return torch.from_numpy(d).cuda()

    def codes(c):
        return torch.from_numpy(np.ascontiguousarray(c, np.int8).reshape(pages, 1, PAGE, dim)).cuda()

    return B.KvCache(codes(k), codes(v), steps(dk), steps(dv))


def expected(q, k, v, dk, dv, scale, length, new):
    """(y, lse, bound of y before its rounding, bound of lse) of the last `new` tokens, causal;
    q float64 [new, group, dim]."""
    dim = k.shape[1]
    dk, dv = (np.repeat(np.asarray(d, np.float32).astype(np.float64), BLOCK) for d in (dk, dv))
    y, lse, ty, tl = (np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape),
                      np.zeros(q.shape[:2]))
    v = v.astype(np.float64)
    for i in range(new):
        n = length - new + i + 1
        kk = k[:n].astype(np.float64)
        for h in range(q.shape[1]):
            s = kk @ q[i, h] * dk[:n] * scale
            size = np.abs(kk) @ np.abs(q[i, h]) * dk[:n] * scale
            p = np.exp(s - s.max())
            total = p.sum()
            w = p * dv[:n] / total
            y[i, h] = w @ v[:n]
            lse[i, h] = s.max() + np.log(total)
            e = dim * 2.0**-22 * size.max() + 2.0**-21 * (1 + np.abs(s).max()) + n * 2.0**-24
            ty[i, h] = ((2 * e + 2.0**-11) * (w @ np.abs(v[:n]))
                        + 2.0**-31 * w.max() * np.abs(v[:n]).sum(0))
            tl[i, h] = e + 2.0**-23 * (1 + abs(lse[i, h]))
    return y, lse, ty, tl


def check(got_y, got_lse, want):
    y, lse, ty, tl = want
    got = got_y.double().cpu().numpy().reshape(y.shape)
    err = np.abs(got - y)
    assert np.all(err <= 2.0**-8 * np.abs(y) + ty * (1 + 2.0**-8)), (err / np.abs(y)).max()
    assert np.all(np.abs(got_lse.double().cpu().numpy().reshape(lse.shape) - lse) <= tl)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("jump", [8, 10, 14, 17, 20.5, 22, 24, 26])
def test_a_score_that_jumps_inside_a_step(B, dim, jump):
    """Flat scores, then one token in a later block of the last step that is 2^jump above them: the
    prompt kernel has stored the step's earlier weights by then, and scales them."""
    length, new = 360, 33
    rng = np.random.default_rng(dim)
    tokens = -(-length // PAGE) * PAGE
    k, v = (np.zeros((tokens, dim), np.int8) for _ in range(2))
    v[:] = rng.integers(20, 120, v.shape)
    v[321] = 0                                   # position 65 of the step that begins at 256
    v[321, ::4] = 1
    k[321, 0] = 100
    dk = np.full(tokens // BLOCK, jump / 100, np.float32)
    dv = np.full(tokens // BLOCK, 0.02, np.float32)
    q = np.zeros((new, 1, dim))
    q[..., 0] = 1
    cache = make_cache(B, k, v, dk, dv)
    Q = torch.from_numpy(q).bfloat16().cuda().flatten(1)
    table = ints(np.arange(tokens // PAGE))[None]
    Y, lse = B.bitnet_kv_attention(cache, Q, 1, ints([0, new]), ints([length]), table, new,
                                   scale=LN2, want_lse=True)
    B.bitnet_sync_status()
    check(Y, lse, expected(q, k, v, dk, dv, LN2, length, new))


@pytest.mark.parametrize("depth", [18.0, 22.0, 25.5, 27.0])
@pytest.mark.parametrize("new,batch", [(1, 296), (33, 296)])
def test_small_weights_behind_a_large_one(B, depth, new, batch):
    """A sink: the first token outweighs each of 65535 others by 2^depth and its V codes are 1 where
    theirs are 100, so together they are up to a quarter of the output.  The sequences share their
    pages; 296 of them leave each block of either kernel one whole sequence."""
    length, dim = 65536 + new, 64
    tokens = -(-length // PAGE) * PAGE
    k, v = np.zeros((tokens, dim), np.int8), np.full((tokens, dim), 100, np.int8)
    k[0, 0] = 100
    v[0] = 1
    dk = np.full(tokens // BLOCK, depth / 100, np.float32)
    dv = np.full(tokens // BLOCK, 0.02, np.float32)
    q = np.zeros((new, 1, dim))
    q[..., 0] = 1
    cache = make_cache(B, k, v, dk, dv)
    Q = torch.from_numpy(q).bfloat16().cuda().flatten(1).repeat(batch, 1)
    table = ints(np.arange(tokens // PAGE))[None].repeat(batch, 1)
    Y, lse = B.bitnet_kv_attention(cache, Q, 1, ints(np.arange(batch + 1) * new),
                                   ints([length] * batch), table, new, scale=LN2, want_lse=True)
    B.bitnet_sync_status()
    want = expected(q, k, v, dk, dv, LN2, length, new)
    Y, lse = Y.view(batch, new, dim), lse.view(batch, new)
    for s in {0, batch // 2, batch - 1}:
        check(Y[s], lse[s], want)


@pytest.mark.parametrize("small", [2.0**-16, 2.0**-20, 2.0**-24, 2.0**-28])
@pytest.mark.parametrize("row", [1.0, 2.0**-50, 2.0**60])
@pytest.mark.parametrize("new", [1, 40])
def test_query_features_of_very_different_size(B, small, row, new):
    """One feature of q is far larger than the others, where the keys have zeros: the scores are made
    of the others.  (Both kernels keep bits down to 2^-38 of the row's largest.)"""
    length, dim = 200, 64
    rng = np.random.default_rng(7)
    tokens = 256
    k, v = (rng.integers(-127, 128, (tokens, dim)).astype(np.int8) for _ in range(2))
    k[:, 5] = 0
    q = rng.uniform(1, 2, (new, 1, dim)) * rng.choice([-1, 1], (new, 1, dim))
    q = torch.from_numpy(q).bfloat16()
    q = q * small
    q[..., 5] = 1.5
    q = q * row
    Q = q.cuda().flatten(1)
    dk = np.full(tokens // BLOCK, 0.01 / small / row, np.float32)
    dv = np.full(tokens // BLOCK, 0.02, np.float32)
    cache = make_cache(B, k, v, dk, dv)
    Y, lse = B.bitnet_kv_attention(cache, Q, 1, ints([0, new]), ints([length]),
                                   ints(np.arange(4))[None], new, scale=0.125, want_lse=True)
    B.bitnet_sync_status()
    check(Y, lse, expected(q.double().numpy(), k, v, dk, dv, 0.125, length, new))
