"""Refusals and sizes of the residual norm, K/V cache and attention entries (no GPU needed): every
call here is answered by the host checks."""
import ctypes
import os

import numpy as np
import pytest
import torch

P = 1 << 20   # a pointer that is never dereferenced


@pytest.fixture(scope="module")
def B():
    from bit_activation_linear_b200 import binding, build
    build.build()
    binding.load_library()
    return binding


@pytest.fixture(scope="module")
def lib(B):
    return B.load_library()


def cache(B, **changed):
    f = dict(k_codes=P, v_codes=P, k_scales=P, v_scales=P, num_pages=10, kv_heads=4, head_dim=128,
             page_tokens=64, scale_tokens=16)
    f.update(changed)
    return ctypes.byref(B._CKvCache(**f))


def batch(B, **changed):
    f = dict(q_start=P, kv_len=P, page_table=P, batch=3, max_pages=5, tokens=7)
    f.update(changed)
    return ctypes.byref(B._CKvBatch(**f))


def append(lib, c, b, k=P, ldk=512, v=P, ldv=512):
    return lib.bitnet_kv_cache_append(c, b, k, ldk, v, ldv, None)


def read(lib, c, b, k=P, ldk=512, v=P, ldv=512):
    return lib.bitnet_kv_cache_read(c, b, k, ldk, v, ldv, None)


def attend(lib, c, b, q=P, ldq=1024, heads=8, max_new=1, scale=0.1, y=P, ldy=1024, lse=None,
           ws=P, ws_bytes=1 << 40):
    return lib.bitnet_kv_attention(c, b, q, ldq, heads, max_new, scale, 1, y, ldy, lse, ws,
                                   ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(k_codes=None), -1), (dict(v_scales=None), -1), (dict(v_codes=P + 8), -1),
    (dict(k_scales=P + 2), -1), (dict(num_pages=0), -1), (dict(num_pages=2**31), -1),
    (dict(kv_heads=0), -1), (dict(kv_heads=1025), -1), (dict(head_dim=96), -2),
    (dict(head_dim=0), -2), (dict(page_tokens=8), -2), (dict(page_tokens=48), -2),
    (dict(page_tokens=512), -2), (dict(page_tokens=-64), -2), (dict(scale_tokens=8), -2),
    (dict(scale_tokens=128), -2), (dict(scale_tokens=0), -2)])
def test_caches_that_are_refused(B, lib, change, status):
    for call in (append, read, attend):
        assert call(lib, cache(B, **change), batch(B)) == status
        assert lib.bitnet_last_error().decode()
    assert lib.bitnet_kv_attention_workspace_bytes(cache(B, **change), batch(B), 8, 1) == 0


@pytest.mark.parametrize("change", [
    dict(q_start=None), dict(kv_len=None), dict(page_table=None), dict(kv_len=P + 1),
    dict(batch=-1), dict(batch=2**21), dict(max_pages=0), dict(max_pages=2**26),
    dict(tokens=-1), dict(tokens=2**29)])
def test_batches_that_are_refused(B, lib, change):
    for call in (append, read, attend):
        assert call(lib, cache(B), batch(B, **change)) == -1


def test_null_structures_are_refused(B, lib):
    for call in (append, read, attend):
        assert call(lib, None, batch(B)) == -1
        assert call(lib, cache(B), None) == -1
    assert lib.bitnet_kv_attention_workspace_bytes(None, None, 8, 1) == 0


def test_matrices_that_are_refused(B, lib):
    for call in (append, read):
        for bad in (dict(k=None), dict(v=None), dict(k=P + 8), dict(ldk=504), dict(ldv=513),
                    dict(ldv=-512), dict(ldk=2**33)):
            assert call(lib, cache(B), batch(B), **bad) == -1
    for bad in (dict(q=None), dict(y=None), dict(q=P + 2), dict(y=P + 8), dict(ldq=1020),
                dict(ldy=1016), dict(heads=0), dict(heads=6), dict(heads=4 * 129), dict(heads=-4),
                dict(max_new=0), dict(max_new=-1), dict(max_new=2**29), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(lse=P + 2)):
        assert attend(lib, cache(B), batch(B), **bad) == -1, bad


def test_more_rows_than_a_launch_holds_are_refused(B, lib):
    big = batch(B, tokens=2**28)
    assert attend(lib, cache(B, kv_heads=1024), big, heads=128 * 1024, ldq=2**24, ldy=2**24) == -2
    assert lib.bitnet_kv_attention_workspace_bytes(cache(B, kv_heads=1024), big, 128 * 1024, 1) == 0


def test_empty_calls_are_answered_without_a_device(B, lib):
    for change in (dict(tokens=0), dict(batch=0, q_start=None, kv_len=None, page_table=None)):
        for call in (append, read, attend):
            assert call(lib, cache(B), batch(B, **change)) == 0


@pytest.mark.parametrize("max_new", [1, 8, 9, 500])
@pytest.mark.parametrize("change", [dict(tokens=0), dict(tokens=0, batch=0), dict(batch=0),
                                    dict(batch=0, tokens=2)])
def test_empty_batches_need_no_workspace(B, lib, change, max_new):
    """Few and many rows (both attention kernels), asked in a child: a signal there is a failure
    here and does not end the run."""
    pid = os.fork()
    if pid == 0:
        need = lib.bitnet_kv_attention_workspace_bytes(cache(B), batch(B, **change), 16, max_new)
        os._exit(need != 0)
    assert os.waitpid(pid, 0)[1] == 0
    assert attend(lib, cache(B), batch(B, **change), heads=16, max_new=max_new, ldq=2048, ldy=2048,
                  ws=None, ws_bytes=0) == 0


def test_attention_workspace_size_and_refusal(B, lib):
    need = lib.bitnet_kv_attention_workspace_bytes(cache(B), batch(B, max_pages=2000), 8, 1)
    assert need % 256 == 0
    if need:
        big = batch(B, max_pages=2000)
        assert attend(lib, cache(B), big, ws_bytes=need - 1) == -5
        assert attend(lib, cache(B), big, ws=None, ws_bytes=need) == -1
        assert attend(lib, cache(B), big, ws=P + 4, ws_bytes=need) == -1


def test_residual_norm_refusals(lib):
    p, q = P, P + 8

    def quant(x=p, r=p, m=4, k=256, gain=None, eps=1e-5, bits=8, h=p, codes=p, scales=p, sums=p):
        return lib.bitnet_act_quant_residual_norm(x, r, m, k, gain, eps, bits, h, codes, scales,
                                                  sums, None)

    def layer(x=p, r=p, m=4, k=256, gain=None, eps=1e-5, bits=8, h=p, y=p, ws=p, ws_bytes=1 << 30):
        return lib.bitnet_residual_norm_bitlinear_forward(x, r, m, k, gain, eps, p, p, 256, bits,
                                                          h, y, ws, ws_bytes, None)

    for bad in (dict(x=None), dict(r=None), dict(h=None), dict(x=q), dict(r=q), dict(h=q),
                dict(m=0), dict(k=200), dict(k=0), dict(bits=3), dict(eps=0.0),
                dict(eps=float("nan")), dict(gain=q)):
        assert quant(**bad) == -1, bad
        assert layer(**bad) == -1, bad
    for bad in (dict(codes=None), dict(codes=q), dict(scales=None), dict(sums=None)):
        assert quant(**bad) == -1
    assert layer(y=None) == -1 and layer(ws=None) == -1
    assert layer(ws_bytes=100) == -5


def test_binding_refuses_what_the_library_cannot_see(B):
    one = torch.zeros((2, 2, 16, 64), dtype=torch.int8)
    steps = torch.zeros((2, 2, 1))
    with pytest.raises(ValueError, match="CUDA"):
        B.KvCache(one, one, steps, steps)
    with pytest.raises(ValueError, match="scale_tokens"):
        B.KvCache.empty(2, 2, 64, page_tokens=64, scale_tokens=24, device="cpu")
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.bitnet_act_quant_residual_norm(x, x, None, 1e-5, 8)
    with pytest.raises(ValueError, match="CUDA"):
        B._rows(x, "Q", 256, None, 0)
    with pytest.raises(TypeError):
        B._rows([1], "Q", 256, None, 0)


def test_rows_of_one_head_in_any_layout(B):
    """[tokens, heads, head_dim] with one head (or one token): the distance of the heads (of the rows)
    means nothing then and may be anything."""
    wide = torch.zeros((1, 6, 256), dtype=torch.bfloat16)
    one_head = wide[:, :, 64:128].transpose(0, 1)
    assert one_head.shape == (6, 1, 64) and not one_head.is_contiguous()
    assert B._rows(one_head, "K", 64, 6, -1) == (one_head.data_ptr(), 256)
    one_token = torch.zeros((4, 2, 64), dtype=torch.bfloat16)[2:3]
    assert B._rows(one_token, "K", 128, 1, -1) == (one_token.data_ptr(), 128)
    heads = torch.zeros((6, 4, 64), dtype=torch.bfloat16)
    assert B._rows(heads[:, 1:3], "K", 128, 6, -1) == (heads.data_ptr() + 128, 256)
    with pytest.raises(ValueError, match="one after the other"):
        B._rows(heads[:, ::2], "K", 128, 6, -1)
    with pytest.raises(ValueError, match="one after the other"):
        B._rows(heads[:, :, ::2], "K", 128, 6, -1)


def test_no_rows_in_any_layout(B):
    """A matrix of no tokens has no distances (numpy's empty arrays come with other strides)."""
    for t, width in ((torch.from_numpy(np.zeros((0, 64), np.float32)).bfloat16(), 64),
                     (torch.empty((4, 64), dtype=torch.bfloat16)[:0].as_strided((0, 64), (64, 2)), 64),
                     (torch.empty(4, dtype=torch.bfloat16).as_strided((0, 2, 64), (1, 0, 7)), 128)):
        assert t.shape[0] == 0 and t.stride()[-1] != 1
        assert B._rows(t, "Q", width, 0, -1)[1] == width
