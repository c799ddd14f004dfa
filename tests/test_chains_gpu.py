"""Forwards one after the other on shared buffers, with nothing that waits between them: every call
gives what it gives alone.

The product is launched while its quantiser still runs (programmatic launch), and the next call's
quantiser writes the codes, scales and code sums to the places of this one's.  Eagerly and in a
replayed graph, as a decoding loop runs them.
"""
import numpy as np
import pytest
import torch

from bit_activation_linear_b200 import synth

pytestmark = pytest.mark.gpu

CALLS = 8


@pytest.fixture(scope="module")
def B():
    from bit_activation_linear_b200 import build, binding
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load_library()
    return binding


def inputs(M, K):
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    return [torch.randn((M, K), generator=gen, device="cuda").bfloat16() for _ in range(CALLS)]


def check_chain(xs, call, out):
    """call(x) writes `out`: alone, in an eager chain and in a replayed one."""
    want = []
    for x in xs:
        torch.cuda.synchronize()
        call(x)
        torch.cuda.synchronize()
        want.append(out.clone())
    for i in range(1, CALLS):
        assert not torch.equal(want[0], want[i])   # another call's result would show
    got = [torch.empty_like(out) for _ in xs]

    def chain():
        for x, g in zip(xs, got):
            call(x)
            g.copy_(out)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for run in [graph.replay] * 10 + [chain] * 10:
        for g in got:
            g.zero_()
        run()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hadamard", [False, True])
@pytest.mark.parametrize("M", [1, 2, 4, 8, 9, 64, 200])
@pytest.mark.parametrize("K,N", [(2048, 512), (256, 2048), (8192, 8192)])
def test_chains_of_forwards(B, M, hadamard, bits, K, N):
    Wp, gamma = B.bitnet_quantize_pack_weights(
        synth.to_torch_bf16(synth.latent_weights(N, K, seed=K)).cuda())
    Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.bitnet_workspace_bytes(M, K, N, bits), dtype=torch.uint8, device="cuda")
    forward = B.bitnet_hbitlinear_forward if hadamard else B.bitnet_bitlinear_forward
    check_chain(inputs(M, K), lambda x: forward(x, Wp, gamma, bits, Y=Y, ws=ws), Y)
    B.bitnet_sync_status()


@pytest.mark.parametrize("M", [1, 5, 8])
@pytest.mark.parametrize("hadamard", [False, True])
@pytest.mark.parametrize("activation", [0, 1, 2])
def test_chains_of_base3_forwards(B, M, hadamard, activation):
    K, N = 2048, 1024
    Wp3, gamma = B.bitnet_quantize_pack_weights_base3(
        synth.to_torch_bf16(synth.latent_weights(N, K, seed=K)).cuda())
    Y = torch.empty((M, N // 2 if activation == 2 else N), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.bitnet_workspace_bytes(M, K, N, 8), dtype=torch.uint8, device="cuda")
    check_chain(inputs(M, K), lambda x: B.bitnet_bitlinear_forward_base3(
        x, Wp3, gamma, hadamard, activation, Y=Y, ws=ws), Y)
    B.bitnet_sync_status()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_chains_of_residual_norm_forwards(B, M, bits):
    """The residual stream is the previous call's H, in place."""
    K, N = 2048, 1024
    Wp, gamma = B.bitnet_quantize_pack_weights(
        synth.to_torch_bf16(synth.latent_weights(N, K, seed=K)).cuda())
    Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.bitnet_workspace_bytes(M, K, N, bits), dtype=torch.uint8, device="cuda")
    H = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    xs = inputs(M, K)

    def call(x):
        if x is xs[0]:
            H.zero_()
        B.bitnet_residual_norm_bitlinear_forward(x, H, None, 1e-5, Wp, gamma, bits, H=H, Y=Y, ws=ws)

    check_chain(xs, call, Y)
    B.bitnet_sync_status()


@pytest.mark.parametrize("M", [1, 8, 40])
def test_chains_of_layers_that_feed_one_another(B, M):
    """A layer's output is the next one's input: norm and up projection, Hadamard and down projection,
    on one workspace."""
    K, F = 1024, 4096
    up, gu = B.bitnet_quantize_pack_weights(
        synth.to_torch_bf16(synth.latent_weights(F, K, seed=1)).cuda())
    down, gd = B.bitnet_quantize_pack_weights(
        synth.to_torch_bf16(synth.latent_weights(K, F, seed=2)).cuda())
    need = max(B.bitnet_workspace_bytes(M, K, F, 8), B.bitnet_workspace_bytes(M, F, K, 8))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")

    def call(x):
        for i in range(4):
            B.bitnet_norm_bitlinear_forward(x if i == 0 else y, None, 1e-5, False, up, gu, 8, Y=a,
                                            ws=ws)
            B.bitnet_hbitlinear_forward(a, down, gd, 8, Y=y, ws=ws)

    check_chain(inputs(M, K), call, y)
    B.bitnet_sync_status()


@pytest.mark.parametrize("hadamard", [False, True])
@pytest.mark.parametrize("base3,M", [(False, 1), (False, 8), (False, 16), (False, 64), (False, 128),
                                     (True, 1), (True, 8)])
@pytest.mark.parametrize("K,N", [(256, 256), (8192, 2048), (16384, 512)])
def test_chains_of_weights_and_forwards(B, M, hadamard, base3, K, N):
    """Weights quantised into the same place right before each forward: the product may load them
    before it waits for its own quantiser, not before they are there."""
    ws = torch.empty(B.bitnet_workspace_bytes(M, K, N, 8), dtype=torch.uint8, device="cuda")
    weights = [synth.to_torch_bf16(synth.latent_weights(N, K, seed=i)).cuda() for i in range(CALLS)]
    pack = B.bitnet_quantize_pack_weights_base3 if base3 else B.bitnet_quantize_pack_weights
    Wp, gamma = pack(weights[0])
    Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    wws = torch.empty(max(256, B.bitnet_weight_workspace_bytes(N, K)), dtype=torch.uint8,
                      device="cuda")
    x = inputs(M, K)[0]

    def call(W):
        pack(W, Wp, gamma, ws=wws)
        if base3:
            B.bitnet_bitlinear_forward_base3(x, Wp, gamma, hadamard, 0, Y=Y, ws=ws)
        elif hadamard:
            B.bitnet_hbitlinear_forward(x, Wp, gamma, 8, Y=Y, ws=ws)
        else:
            B.bitnet_bitlinear_forward(x, Wp, gamma, 8, Y=Y, ws=ws)

    check_chain(weights, call, Y)
    B.bitnet_sync_status()


def test_forwards_from_several_host_threads(B):
    """The first calls of several quantisers and products from eight threads at once, a stream each,
    give what they give one after the other."""
    import threading

    jobs = []
    for K in (128, 512, 1024, 4096, 16384):
        W = synth.to_torch_bf16(synth.latent_weights(256, K, seed=K)).cuda()
        jobs += [(K, M, bits, *B.bitnet_quantize_pack_weights(W)) for M in (1, 20, 100)
                 for bits in (8, 4)]

    def work(stream, out):
        with torch.cuda.stream(stream):
            for K, M, bits, Wp, gamma in jobs:
                x = torch.randn((M, K), generator=torch.Generator(device="cuda").manual_seed(K),
                                device="cuda").bfloat16()
                out.append(B.bitnet_norm_bitlinear_forward(x, None, 1e-5, True, Wp, gamma, bits))
                out.append(B.bitnet_hbitlinear_forward(x, Wp, gamma, bits))
                out.append(B.bitnet_bitlinear_forward(x, Wp, gamma, bits))
            stream.synchronize()

    torch.cuda.synchronize()
    outs = [[] for _ in range(8)]
    threads = [threading.Thread(target=work, args=(torch.cuda.Stream(), out)) for out in outs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    want = []
    work(torch.cuda.current_stream(), want)
    for out in outs:
        assert len(out) == len(want) and all(torch.equal(x, y) for x, y in zip(out, want))
    B.bitnet_sync_status()
