"""The operators that are launched before the kernel in front of them has
ended, in streams that fork and join: eager, and captured, where a kernel's
predecessors are kernels of several streams, copies or fills.  Every result
must be what the calls give one by one."""
import pytest
import torch

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


def _block(F, seed, tokens, states):
    """(inputs, run): Q on the caller's stream, K and V on a second one, joined for the attention; the next
    layer's quantizer after a copy, its GEMM after a fill of another buffer."""
    g = torch.Generator().manual_seed(seed)
    heads, D = 6, 64
    hidden = heads * D
    x = torch.randn(tokens, hidden, generator=g).bfloat16().cuda()
    s = torch.randn(states, hidden, generator=g).bfloat16().cuda()
    wq, wkv, wo = (F.quantize_mxfp4(torch.randn(n, hidden, generator=g).mul(0.05).bfloat16().cuda())
                   for n in (hidden, 2 * hidden, hidden))
    pos_q, pos_k = (torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous() for n in (tokens, states))
    side = torch.cuda.Stream()

    def run(sync=lambda: None):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            sq = F.quantize_mxfp4(s)
            sync()
            kv = F.gemm_mxfp4(sq, wkv).view(1, states, 2, heads, D)
            sync()
            k = F.rope(kv[:, :, 0], pos_k, [D])
            sync()
        xq = F.quantize_mxfp4(x)
        sync()
        q = F.rope(F.gemm_mxfp4(xq, wq).view(1, tokens, heads, D), pos_q, [D])
        sync()
        main.wait_stream(side)
        for t in (sq.codes, sq.sf, kv, k):
            t.record_stream(main)
        o = F.cross_attention(q, k, kv[:, :, 1])
        sync()
        copied = torch.empty_like(o)
        copied.copy_(o)
        oq = F.quantize_mxfp4(copied.view(tokens, hidden))
        sync()
        y = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
        y.zero_()
        F.gemm_mxfp4(oq, wo, y=y)
        sync()
        return y, o

    return (x, s), run


@pytest.mark.parametrize("tokens,states", [(1, 1500), (300, 77), (1500, 700)])
def test_forks_and_joins(F, tokens, states):
    (x, s), run = _block(F, tokens, tokens, states)
    want = run(torch.cuda.synchronize)
    for _ in range(5):
        got = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for scale in (1.0, -2.0):
        x.mul_(scale)
        s.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        one_by_one = run(torch.cuda.synchronize)
        assert all(torch.equal(a, b) for a, b in zip(got, one_by_one))
    F.nvfp4_check_fault()


def test_two_graphs_at_once(F):
    blocks = [_block(F, seed, *n) for seed, n in ((1, (300, 900)), (2, (40, 2000)))]
    want = [run(torch.cuda.synchronize) for _, run in blocks]
    graphs, results = [], []
    for _, run in blocks:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            results.append(run())
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for graph, stream in zip(graphs, streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for got, w in zip(results, want):
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    F.nvfp4_check_fault()
