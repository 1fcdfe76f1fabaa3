"""The operators of an attention block in the order a model runs them: MXFP4
projections of the tokens (Q) and of the encoder's states (K and V in one),
rotary positions with the heads' norms in place on the Q columns, attention
over the valid states, MXFP4 output projection.  Each step is checked against
the oracle applied to the step before as the GPU left it, and the whole run,
captured into a graph, against itself on other inputs."""
import numpy as np
import pytest
import torch

import synth
from oracle import heads_ref as H
from oracle import mxfp4_ref as X
from tests.gpu_helpers import assert_bytes_equal, assert_within_tol, f32, gpu_bytes, require_gpu
from tests.test_gpu_attention import _check as check_attention
from tests.test_gpu_rope import _check as check_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


def _check_linear(F, x, xq, w, y, bias):
    a_codes, a_sf = X.quantize_mxfp4(f32(x.cpu()))
    assert_bytes_equal(gpu_bytes(xq.codes), a_codes, "codes")
    assert_bytes_equal(gpu_bytes(xq.sf), X.swizzle_sf_mxfp4(a_sf), "scales")
    b_codes, b_sf = X.quantize_mxfp4(f32(w))
    y_ref = X.gemm_ref_mxfp4(a_codes, a_sf, b_codes, b_sf, 1.0, f32(bias))
    assert_within_tol(y.float().cpu().numpy(), y_ref, X.gemm_tolerance_mxfp4(a_codes, a_sf, b_codes, b_sf, y_ref), "y")


@pytest.mark.parametrize("B,L,Lk,heads,D", [(1, 1, 50, 4, 64), (2, 130, 77, 3, 128), (2, 96, 300, 8, 64)])
def test_attention_block(F, B, L, Lk, heads, D):
    K, hidden, states_k = 320, heads * D, 192
    x = synth.activations_with_outlier_channels(B * L, K, seed=L).cuda()
    states = synth.activations_with_outlier_channels(B * Lk, states_k, seed=Lk).cuda()
    gen = synth._gen(3)
    w_q, w_kv, w_o = (synth.normal_bf16(s, 0.05, gen) for s in ((hidden, K), (2 * hidden, states_k), (256, hidden)))
    b_q, b_kv, b_o = (synth.normal_bf16((n,), 0.1, gen) for n in (hidden, 2 * hidden, 256))
    norm = (1 + synth.normal_bf16((D,), 0.2, gen).float()).bfloat16().cuda()
    wq, wkv, wo = (F.quantize_mxfp4(w.cuda()) for w in (w_q, w_kv, w_o))
    bq, bkv, bo = (b.cuda() for b in (b_q, b_kv, b_o))
    lens = torch.tensor([Lk, Lk // 3][:B], dtype=torch.int32).cuda()
    pos = torch.randint(0, 40, (L, 3), dtype=torch.int32).cuda()
    axes = [D // 4, 3 * D // 8, 3 * D // 8]
    steps = {}

    def run():
        xq, sq = F.quantize_mxfp4(x), F.quantize_mxfp4(states)
        q = F.gemm_mxfp4(xq, wq, bias=bq)
        kv = F.gemm_mxfp4(sq, wkv, bias=bkv)
        turned = F.rope(q.view(B, L, heads, D), pos, axes, q_weight=norm)
        k, v = kv.view(B, Lk, 2, heads, D).unbind(2)
        o = F.cross_attention(turned, k, v, kv_lens=lens)
        oq = F.quantize_mxfp4(o.view(B * L, hidden))
        y = F.gemm_mxfp4(oq, wo, bias=bo)
        steps.update(xq=xq, sq=sq, q=q, kv=kv, turned=turned, k=k, v=v, o=o, oq=oq, y=y)
        return y

    run()
    torch.cuda.synchronize()
    s = steps
    _check_linear(F, x, s["xq"], w_q, s["q"], b_q)
    _check_linear(F, states, s["sq"], w_kv, s["kv"], b_kv)
    check_rope(s["turned"], s["q"].view(B, L, heads, D), pos, axes, "rope", weight=norm)
    check_attention(s["o"], s["turned"], s["k"], s["v"], lens)
    _check_linear(F, s["o"].view(B * L, hidden), s["oq"], w_o, s["y"], b_o)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        captured = run()
    x.mul_(-1.5)
    lens.copy_(lens.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    replayed = captured.clone()
    assert torch.equal(replayed, run())
    F.nvfp4_check_fault()


def _calls(F, seed):
    """The operators on inputs of their own, at sizes that take clusters, pairs and one-CTA tiles, and their results
    when nothing else runs."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    q, k, v = rand(2, 5, 8, 128), rand(2, 3000, 4, 128), rand(2, 3000, 4, 128)
    lens = torch.tensor([3000, 1234], dtype=torch.int32).cuda()
    big = rand(1, 900, 12, 64), rand(1, 300, 12, 64), rand(1, 300, 12, 64)
    pos = torch.randint(0, 99, (900, 2), dtype=torch.int32).cuda()
    weights = [F.quantize_mxfp4(rand(n, 448)) for n in (520, 1024)]
    xs = [rand(m, 448) for m in (1, 300, 3000)]

    def run():
        out = [F.cross_attention(q, k, v, kv_lens=lens), F.cross_attention(*big), F.rope(big[0], pos, [32, 32])]
        for x in xs:
            for w in weights:
                out.append(F.gemm_mxfp4(F.quantize_mxfp4(x), w))
        return out

    return run


def test_streams_and_host_threads_at_once(F):
    from concurrent.futures import ThreadPoolExecutor
    runs = [_calls(F, seed) for seed in range(4)]
    want = [run() for run in runs]
    torch.cuda.synchronize()

    def worker(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [runs[i]() for _ in range(5)]
        stream.synchronize()
        return got

    with ThreadPoolExecutor(4) as pool:
        for i, rounds in enumerate(pool.map(worker, range(4))):
            for got in rounds:
                for a, b in zip(got, want[i]):
                    assert torch.equal(a, b)
    F.nvfp4_check_fault()


def test_outputs_given_nothing_is_allocated(F):
    q, k = torch.randn(1, 40, 4, 64, device="cuda").half(), torch.randn(1, 2000, 2, 64, device="cuda").half()
    x, w = torch.randn(70, 192, device="cuda").bfloat16(), F.quantize_mxfp4(torch.randn(64, 192, device="cuda").bfloat16())
    pos = torch.zeros(40, 1, dtype=torch.int32, device="cuda")
    xq, y, o = F.quantize_mxfp4(x), torch.empty(70, 64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(q)

    def run():
        F.quantize_mxfp4(x, out=xq)
        F.gemm_mxfp4(xq, w, y=y)
        F.rope(q, pos, [64], q_out=o)
        F.cross_attention(q, k, k, out=o)

    run()
    torch.cuda.synchronize()
    before, free = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
    run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert torch.cuda.mem_get_info()[0] == free


@pytest.mark.parametrize("L", [1, 700])
def test_calls_in_a_row_equal_calls_one_by_one(F, L):
    # each kernel sets itself up while the one in front of it ends; every call reads what the last one wrote, into
    # buffers that the last but one read
    heads, D = 8, 64
    gen = torch.Generator("cuda").manual_seed(3)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen).to(torch.bfloat16)  # noqa: E731
    x0, k, v = rand(L, heads * D), rand(1, 1500, heads, D), rand(1, 1500, heads, D)
    w = F.quantize_mxfp4(rand(heads * D, heads * D) * 0.1)
    pos = torch.arange(2 * L, device="cuda", dtype=torch.int32).view(L, 2)

    def run(sync):
        x, y, xq = x0.clone(), torch.empty_like(x0), None
        turned, o = (torch.empty(1, L, heads, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        for _ in range(30):
            xq = F.quantize_mxfp4(x, out=xq)
            sync()
            F.gemm_mxfp4(xq, w, y=y)
            sync()
            F.rope(y.view(1, L, heads, D), pos, [32, 32], q_out=turned)
            sync()
            F.rope(turned, pos, [32, 32], q_out=turned)
            sync()
            F.cross_attention(turned, k, v, out=o)
            sync()
            F.cross_attention(o, k, v, out=x.view(1, L, heads, D))
            sync()
            x.add_(x0)
            sync()
        return x

    one_by_one = run(torch.cuda.synchronize)
    for _ in range(3):
        assert torch.equal(run(lambda: None), one_by_one)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(lambda: None)
    graph.replay()
    assert torch.equal(got, one_by_one)
    F.nvfp4_check_fault()
