"""GPU parity of attention over states of another length against the float64
oracle.

Tolerance, with h = eps / 2 of the type, n valid keys, w = sum p |v| / sum p
and a = scale * max |q| |k| over the row's keys (2-norms):
  * P is rounded once: a relative h on every probability, so h w;
  * a probability's exponent carries the score's fp32 sum (2^-23 a per addition
    of D: D 2^-23 a) and its own arithmetic (8 a 2^-24), and exp2 adds 2^-22:
    the numerator's and the denominator's, so twice that times w;
  * the fp32 sums over n keys: 2 n 2^-23 w;
  * fp16 probabilities below 2^-14 round by 2^-25 absolutely, against a sum of
    at least 1: n 2^-25 max |v|;
  * the result is rounded once: h |o| (half of fp16's smallest step 2^-25)."""
import numpy as np
import pytest
import torch

from oracle import heads_ref as H
from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(o, q, k, v, lens=None, scale=None, what=""):
    D, Lk = q.shape[3], k.shape[1]
    c = 1.0 / np.sqrt(D) if scale is None else scale
    n_valid = np.full(q.shape[0], Lk) if lens is None else np.clip(_np(lens).astype(int), 0, Lk)
    kk, vv = _np(k).copy(), _np(v).copy()
    for b, n in enumerate(n_valid):  # what lies behind the valid states is nobody's business
        kk[b, n:], vv[b, n:] = 0.0, 0.0
    want, w = H.attention_ref(_np(q), kk, vv, n_valid, c)
    h = torch.finfo(o.dtype).eps / 2
    a = c * np.linalg.norm(_np(q), axis=3, keepdims=True).max() * np.linalg.norm(kk, axis=3).max()
    n = max(1, n_valid.max())
    tol = w * (h + 2 * (D * 2.0 ** -23 * a + 8 * a * 2.0 ** -24 + 2.0 ** -22) + 2 * n * 2.0 ** -23) + h * np.abs(want)
    if o.dtype == HF:
        tol = tol + 2.0 ** -25 * (1 + n * np.abs(vv).max())
    err = np.abs(_np(o) - want)
    bad = np.argwhere(~(err <= tol * 1.001))
    assert bad.size == 0, f"{what}: {len(bad)} of {err.size} off, first {bad[0]}: {_np(o)[tuple(bad[0])]} " \
                          f"for {want[tuple(bad[0])]}, tolerance {tol[tuple(bad[0])]}"


# Whole items in turn, fewer and more of them than SMs; items with CTAs of their own: keys split over clusters of up
# to 8, one query tile whose two slots take the key tiles in turn, both, and parts without keys
SHAPES = [  # B, Lq, Lk, Hq, Hk, D, dtype
    (1, 1, 1, 1, 1, 8, BF), (1, 1, 1, 1, 1, 128, HF), (1, 128, 128, 1, 1, 64, BF), (1, 129, 129, 1, 1, 128, BF),
    (1, 1, 129, 2, 1, 64, HF), (2, 257, 513, 4, 4, 128, BF), (2, 333, 77, 5, 5, 72, HF), (3, 300, 1000, 6, 2, 96, BF),
    (1, 100, 700, 24, 8, 128, HF), (2, 64, 31, 7, 1, 40, BF), (1, 3, 300, 128, 1, 64, BF), (1, 7, 260, 100, 1, 128, BF),
    (1, 256, 2048, 2, 2, 64, HF), (1, 1, 4095, 8, 1, 128, BF), (2, 1, 5000, 4, 4, 128, HF), (1, 40, 1100, 3, 3, 56, BF),
    (1, 300, 1500, 2, 2, 128, BF), (1, 700, 2000, 9, 3, 64, HF), (5, 1, 2600, 16, 16, 64, BF), (8, 64, 1400, 20, 20, 128, HF),
    (1, 128, 10000, 1, 1, 128, BF), (3, 2, 9000, 21, 7, 88, BF), (20, 3, 400, 16, 8, 64, HF),
    (4, 1000, 200, 8, 8, 128, BF), (4, 700, 300, 16, 16, 64, HF), (2, 1000, 640, 24, 8, 120, BF),
]


@pytest.mark.parametrize("B,Lq,Lk,Hq,Hk,D,dtype", SHAPES)
def test_shapes(F, B, Lq, Lk, Hq, Hk, D, dtype):
    q = _rand((B, Lq, Hq, D), dtype, Lq)
    kv = _rand((B, Lk, 2, Hk, D), dtype, Lk + 1)
    k, v = kv[:, :, 0], kv[:, :, 1]
    o = F.cross_attention(q, k, v)
    assert o.shape == q.shape and o.dtype == dtype and o.is_contiguous()
    _check(o, q, k, v)
    assert torch.equal(o, F.cross_attention(q, k, v))  # the same bits again


# queries of up to 32 rows a K/V head (tokens x heads) over keys that are shared out, and the first shapes past that
@pytest.mark.parametrize("B,Lq,Lk,Hq,Hk,D,dtype", [
    (1, 1, 1025, 1, 1, 128, BF), (2, 32, 1500, 2, 2, 64, HF), (2, 33, 1500, 2, 2, 64, HF), (3, 4, 1700, 40, 5, 128, BF),
    (1, 10, 3000, 3, 1, 72, BF), (2, 6, 5130, 5, 1, 8, HF), (1, 1, 2049, 32, 1, 128, HF), (1, 1, 2049, 33, 1, 128, HF),
    (1, 2, 40000, 16, 1, 128, BF), (40, 1, 1900, 8, 8, 64, BF), (25, 3, 1300, 28, 7, 112, HF), (1, 31, 1111, 1, 1, 24, BF)])
def test_few_queries(F, B, Lq, Lk, Hq, Hk, D, dtype):
    test_shapes(F, B, Lq, Lk, Hq, Hk, D, dtype)


@pytest.mark.parametrize("Lq,Hq,Hk,D,dtype", [(1, 8, 2, 128, BF), (5, 6, 1, 64, HF)])
@pytest.mark.parametrize("rubbish", [float("nan"), float("-inf")])
def test_few_queries_over_states_of_many_lengths(F, Lq, Hq, Hk, D, dtype, rubbish):
    lens = [0, 1, 31, 32, 33, 64, 95, 97, 127, 128, 129, 160, 1000, 1030, 1499, 1500]
    q, k, v = _rand((16, Lq, Hq, D), dtype, 21), _rand((16, 1500, Hk, D), dtype, 22), _rand((16, 1500, Hk, D), dtype, 23)
    for b, n in enumerate(lens):
        k[b, n:] = rubbish
        v[b, n:] = rubbish
    lens = torch.tensor(lens, dtype=torch.int32).cuda()
    o = F.cross_attention(q, k, v, kv_lens=lens)
    _check(o, q, k, v, lens)
    assert bool((o[0] == 0).all())


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 143, 144, 255, 256, 300, 301, 2 ** 31 - 1, -5]


@pytest.mark.parametrize("Lq,Hq,Hk,D,dtype", [(1, 4, 2, 128, BF), (200, 2, 2, 64, HF), (300, 8, 8, 128, BF)])
@pytest.mark.parametrize("rubbish", [float("nan"), float("inf"), float("-inf"), 3e4])
def test_valid_lengths_and_what_lies_behind_them(F, Lq, Hq, Hk, D, dtype, rubbish):
    B, Lk = len(LENS), 301
    q = _rand((B, Lq, Hq, D), dtype, 1)
    k, v = _rand((B, Lk, Hk, D), dtype, 2), _rand((B, Lk, Hk, D), dtype, 3)
    lens = torch.tensor(LENS, dtype=torch.int64).clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32).cuda()
    for b, n in enumerate(LENS):
        k[b, max(0, min(n, Lk)):] = rubbish
        v[b, max(0, min(n, Lk)):] = rubbish
    o = F.cross_attention(q, k, v, kv_lens=lens)
    _check(o, q, k, v, lens)
    assert bool((o[0] == 0).all()) and bool((o[-1] == 0).all())


@pytest.mark.parametrize("Lq,Lk", [(1, 2000), (300, 700), (3000, 300)])
def test_a_scale_and_scores_that_grow_from_tile_to_tile(F, Lq, Lk):
    # every tile's maximum beats the last one's by far more than 2^8 in P for some rows, falls for others
    q = _rand((1, Lq, 4, 64), BF, 4)
    k = _rand((1, Lk, 4, 64), BF, 5)
    ramp = torch.linspace(-3, 3, Lk, device="cuda")[None, :, None, None]
    k = (k * 0.2 + ramp * torch.sign(torch.linspace(-1, 1, 64, device="cuda"))).to(BF)
    v = _rand((1, Lk, 4, 64), BF, 6)
    o = F.cross_attention(q, k, v, scale=0.7)
    _check(o, q, k, v, scale=0.7)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64), (BF, 72)])
@pytest.mark.parametrize("Lq,Lk", [(1, 1500), (130, 1500), (1500, 130)])
def test_one_key_takes_everything_bit_exact(F, dtype, D, Lq, Lk):
    # query t points at key (7 t) mod Lk: its score leads by more than 150 binary orders, so P is 1 there and 0
    # elsewhere and the result is that key's V, bit for bit, wherever it lies
    code = ((torch.arange(Lk, device="cuda")[:, None] >> torch.arange(11, device="cuda")) & 1) * 2 - 1
    k = torch.zeros(1, Lk, 2, D, device="cuda", dtype=dtype)
    k[0, :, :, :11] = code[:, None].to(dtype)
    v = _rand((1, Lk, 2, D), dtype, 8)
    pick = (torch.arange(Lq, device="cuda") * 7) % Lk
    q = torch.zeros(1, Lq, 2, D, device="cuda", dtype=dtype)
    q[0, :, :, :11] = code[pick][:, None].to(dtype) * 64
    o = F.cross_attention(q, k, v, scale=1.0)
    assert torch.equal(o[0], v[0, pick])


@pytest.mark.parametrize("Lq,Lk,inf_to", [(1, 600, 400), (200, 600, 400), (200, 300, 130), (1, 300, 300), (200, 300, 300)])
def test_scores_of_minus_infinity(F, Lq, Lk, inf_to):
    # a valid state whose key holds -inf (and queries that are positive there) has a probability of zero; the first
    # tiles have nothing else, and the last two cases no finite score at all
    q, k, v = (_rand((1, n, 4, 64), BF, 40 + n) for n in (Lq, Lk, Lk))
    q[..., 0] = 1.0
    k[:, :inf_to, :, 0] = float("-inf")
    o = F.cross_attention(q, k, v)
    if inf_to == Lk:
        assert bool((o == 0).all())
    else:
        _check(o, q, k[:, inf_to:], v[:, inf_to:])


def test_a_score_that_is_not_a_number_shows(F):
    for Lq in (1, 200):
        q, k, v = (_rand((1, n, 4, 64), BF, 50 + n) for n in (Lq, 600, 600))
        k[0, 300, 1, 5] = float("nan")
        o = F.cross_attention(q, k, v)
        assert bool(torch.isnan(o[:, :, 1]).all()) and not bool(torch.isnan(o[:, :, [0, 2, 3]]).any())


@pytest.mark.parametrize("Lq,Lk", [(1, 200), (1, 3000), (200, 600), (3000, 300)])
def test_a_query_that_is_not_a_number_shows(F, Lq, Lk):
    # (keys in one CTA's hands and split over several)
    q, k, v = (_rand((1, n, 4, 64), BF, 60 + n) for n in (Lq, Lk, Lk))
    q[0, Lq // 2, 1, 5] = float("nan")
    bad = torch.zeros(1, Lq, 4, 64, dtype=torch.bool, device="cuda")
    bad[0, Lq // 2, 1] = True
    assert torch.equal(torch.isnan(F.cross_attention(q, k, v)), bad)


def test_equal_scores_give_the_mean(F):
    q = torch.zeros(2, 50, 2, 128, device="cuda", dtype=BF)
    k, v = _rand((2, 512, 2, 128), BF, 9), torch.ones(2, 512, 2, 128, device="cuda", dtype=BF)
    assert bool((F.cross_attention(q, k, v) == 1).all())
    lens = torch.tensor([333, 1], dtype=torch.int32).cuda()
    v[1] = _rand((512, 2, 128), BF, 10)
    o = F.cross_attention(q, k, v, kv_lens=lens)
    assert bool((o[0] == 1).all()) and torch.equal(o[1], v[1, :1].expand(50, 2, 128))


def test_views_of_fused_projections_and_padded_outputs(F):
    B, Lq, Lk, Hq, Hk, D = 2, 150, 90, 6, 3, 64
    qkv = _rand((B, Lq, (Hq + 2 * Hk) * D + 64), BF, 11)
    q = qkv[:, :, :Hq * D].unflatten(2, (Hq, D))
    kv = _rand((B, 2 * Hk, Lk, D), BF, 12)  # heads before tokens
    k, v = kv[:, :Hk].transpose(1, 2), kv[:, Hk:].transpose(1, 2)
    store = torch.full((B, Lq + 1, Hq, 72), 7.0, device="cuda", dtype=BF)
    F.cross_attention(q, k, v, out=store[:, :Lq, :, :D])
    _check(store[:, :Lq, :, :D], q, k, v)
    assert bool((store[:, Lq:] == 7.0).all()) and bool((store[..., D:] == 7.0).all())


def test_states_shared_by_the_batch(F):
    q = _rand((3, 140, 4, 128), BF, 13)
    k1, v1 = _rand((1, 200, 4, 128), BF, 14), _rand((1, 200, 4, 128), BF, 15)
    k, v = k1.expand(3, -1, -1, -1), v1.expand(3, -1, -1, -1)
    lens = torch.tensor([200, 3, 0], dtype=torch.int32).cuda()
    o = F.cross_attention(q, k, v, kv_lens=lens)
    _check(o, q, k, v, lens)
    o = F.cross_attention(q[:1].expand(3, -1, -1, -1), k, v, kv_lens=lens)
    _check(o, q[:1].expand(3, -1, -1, -1), k, v, lens)


def test_offsets_beyond_32_bits(F):
    # 300 states 2^23 elements apart: the last one lies 5 GB behind the first
    big = torch.empty(300 * 2 ** 23, device="cuda", dtype=BF)
    kv = big.view(1, 300, 2 ** 23)[:, :, :4 * 128].unflatten(2, (2, 2, 128))
    kv.copy_(_rand((1, 300, 2, 2, 128), BF, 16))
    q = _rand((1, 60, 2, 128), BF, 17)
    _check(F.cross_attention(q, kv[:, :, 0], kv[:, :, 1]), q, kv[:, :, 0], kv[:, :, 1])
    out = big.view(1, 300, 2 ** 23)[:, :300, 1024:1024 + 256].unflatten(2, (2, 128))
    q = _rand((1, 300, 2, 128), BF, 18)
    F.cross_attention(q, kv[:, :, 0], kv[:, :, 1], out=out)
    _check(out, q, kv[:, :, 0], kv[:, :, 1])


def test_graph_replay_with_other_lengths_and_another_stream(F):
    B, Lq, Lk = 3, 20, 600
    q, k, v = (_rand((B, n, 4, 128), BF, 19 + n) for n in (Lq, Lk, Lk))
    lens = torch.tensor([600, 200, 1], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    want = F.cross_attention(q, k, v, kv_lens=lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = F.cross_attention(q, k, v, kv_lens=lens, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.cross_attention(q, k, v, kv_lens=lens, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lens.copy_(torch.tensor([0, 600, 77], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    _check(out, q, k, v, lens)


def test_no_kernel_reported_a_fault(F):
    torch.cuda.synchronize()
    F.nvfp4_check_fault()
