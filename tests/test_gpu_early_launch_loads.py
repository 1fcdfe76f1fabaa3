"""Lengths and biases written by the kernel right in front of the one that
reads them, which is launched while that one still runs: the rotary kernel
copies them (elements that pass through keep their bits), call after call, and
each call must see what was copied last."""
import pytest
import torch

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


def _copier(F, src, dst):
    """One launch that copies bf16 [n, 8], the last half of heads of 16 (the first half turns by angles of zero)."""
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    n = dst.shape[0]
    return lambda i: F.rope(src[i].view(1, 1, n, 16), pos, [8], q_out=dst.view(1, 1, n, 16))


@pytest.mark.parametrize("Lq,Lk", [(1, 2000), (200, 2000), (2000, 300)])
def test_lengths_from_the_kernel_in_front(F, Lq, Lk):
    B, rounds = 4, 40
    g = torch.Generator().manual_seed(Lq)
    q, k, v = (torch.randn(B, n, 2, 64, generator=g).bfloat16().cuda() for n in (Lq, Lk, Lk))
    lens = torch.randint(0, Lk + 1, (rounds, B), generator=g, dtype=torch.int32).cuda()
    src = torch.zeros(rounds, 1, 16, dtype=torch.bfloat16, device="cuda")
    src.view(torch.int32).view(rounds, 8)[:, 4:] = lens
    dst = torch.zeros(1, 16, dtype=torch.bfloat16, device="cuda")
    now = dst.view(torch.int32).view(8)[4:]
    copy = _copier(F, src, dst)
    want = [F.cross_attention(q, k, v, kv_lens=lens[i].clone()) for i in range(rounds)]

    def run():
        got = []
        for i in range(rounds):
            copy(i)
            got.append(F.cross_attention(q, k, v, kv_lens=now))
        return got

    for _ in range(3):
        got = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    F.nvfp4_check_fault()


@pytest.mark.parametrize("M,K,N", [(1, 4096, 1024), (200, 320, 1024), (700, 320, 4096), (2600, 320, 2560)])
def test_a_bias_from_the_kernel_in_front(F, M, K, N):
    # a K split, one CTA and pair tiles, wide tiles
    rounds = 30
    g = torch.Generator().manual_seed(M)
    x = F.quantize_mxfp4(torch.randn(M, K, generator=g).bfloat16().cuda())
    w = F.quantize_mxfp4(torch.randn(N, K, generator=g).bfloat16().cuda())
    src = torch.randn(rounds, N // 16, 16, generator=g).bfloat16().cuda()
    bias = torch.zeros(N // 16, 16, dtype=torch.bfloat16, device="cuda")
    copy = _copier(F, src, bias)
    want = [F.gemm_mxfp4(x, w, bias=src[i].reshape(N)) for i in range(rounds)]

    def run():
        got = []
        for i in range(rounds):
            copy(i)
            got.append(F.gemm_mxfp4(x, w, bias=bias.view(N)))
        return got

    for _ in range(3):
        got = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    F.nvfp4_check_fault()
