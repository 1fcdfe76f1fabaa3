"""Attention over valid states that hold infinities, and scores that leave the
range of fp32 once they are scaled: what the definition gives, whichever form
of the kernel the shape takes.

No probability here is small enough to round to zero (scores of unit normal
queries and keys stay within e^-16 of each other, the types hold 2^-25 and
less), so p * inf is inf of its sign for every key, and a column holds +inf,
-inf or, where both meet or a state holds NaN, NaN.  The other columns are
compared with the oracle by the tolerance of the attention tests."""
import numpy as np
import pytest
import torch

from oracle import heads_ref as H
from tests.gpu_helpers import require_gpu
from tests.test_gpu_attention import BF, HF, _check, _np, _rand

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


def _check_classes(o, q, k, v, lens=None):
    """Columns without a finite definition by their class, the others by value."""
    n_valid = [v.shape[1]] * v.shape[0] if lens is None else [int(n) for n in lens.cpu()]
    vv = _np(v).copy()
    for b, n in enumerate(n_valid):
        vv[b, n:] = 0.0
    kk = _np(k).copy()
    for b, n in enumerate(n_valid):
        kk[b, n:] = 0.0
    with np.errstate(invalid="ignore"):
        want, _ = H.attention_ref(_np(q), kk, vv, n_valid, q.shape[3] ** -0.5)
    got = _np(o)
    for name, of in (("nan", np.isnan), ("+inf", np.isposinf), ("-inf", np.isneginf)):
        bad = np.argwhere(of(got) != of(want))
        assert bad.size == 0, f"{name}: {len(bad)} of {got.size} differ, first {bad[0]}: {got[tuple(bad[0])]} " \
                              f"for {want[tuple(bad[0])]}"
    # the finite rest: a K/V head's column with an infinity counts as zeros on both sides
    special = ~np.isfinite(vv).all(axis=1)                                  # [B, Hk, D]
    heads = np.repeat(special, q.shape[2] // k.shape[2], axis=1)            # [B, Hq, D]
    o2 = o.clone()
    o2[torch.from_numpy(heads).cuda()[:, None].expand_as(o2)] = 0.0
    v2 = v.clone()
    v2[torch.from_numpy(special).cuda()[:, None].expand_as(v2)] = 0.0
    _check(o2, q, k, v2, lens)


FORMS = [  # B, Lq, Lk, Hq, Hk, D, dtype
    (3, 1, 1500, 8, 2, 128, BF),    # up to 32 rows a K/V head, keys split over a cluster
    (3, 5, 1500, 6, 1, 64, HF),
    (2, 4, 700, 16, 2, 72, BF),     # 32 rows, a width that is no multiple of 32
    (2, 1, 1030, 7, 7, 8, HF),
    (2, 1, 2000, 20, 1, 128, HF),   # 20 rows, one query
    (2, 33, 1500, 2, 2, 64, HF),    # one more row: the form for whole tiles, joined
    (2, 200, 1500, 2, 2, 128, BF),  # two tiles of queries, joined
    (2, 1500, 130, 6, 2, 64, BF),   # whole items in turn
]


@pytest.mark.parametrize("B,Lq,Lk,Hq,Hk,D,dtype", FORMS)
@pytest.mark.parametrize("with_lens", [False, True])
def test_infinities_in_valid_states(F, B, Lq, Lk, Hq, Hk, D, dtype, with_lens):
    q, k, v = _rand((B, Lq, Hq, D), dtype, 71), _rand((B, Lk, Hk, D), dtype, 72), _rand((B, Lk, Hk, D), dtype, 73)
    lens = None
    n = Lk
    if with_lens:  # rubbish behind the last entry's states, whose last tile ends inside
        n = Lk - 55
        lens = torch.tensor([Lk] * (B - 1) + [n], dtype=torch.int32).cuda()
        k[-1, n:], v[-1, n:] = float("nan"), -INF
    # one key a column, in every quarter of a tile, in first, middle and last tiles
    for col, key in enumerate([0, 31, 33, n // 2]):
        v[:, key, :, col] = INF
    v[:, n - 1, :, 4] = -INF
    v[0, [3, n - 2], 0, 5] = torch.tensor([INF, -INF], device="cuda", dtype=dtype)  # both: NaN
    v[1, 66, -1, 6] = float("nan")
    v[-1, [96, 100], -1, 7] = INF
    o = F.cross_attention(q, k, v, kv_lens=lens)
    _check_classes(o, q, k, v, lens)
    assert torch.equal(o.view(torch.int16), F.cross_attention(q, k, v, kv_lens=lens).view(torch.int16))


def test_an_infinite_column_of_many_states(F):
    # an overflowed projection: every state infinite in one column, half of them in another
    q, k, v = (_rand((2, n, 4, 128), HF, 80 + n) for n in (1, 3000, 3000))
    v[:, :, 1, 17] = INF
    v[:, ::2, 2, 127] = -INF
    _check_classes(F.cross_attention(q, k, v), q, k, v)


def test_infinities_seen_from_a_replayed_graph(F):
    q, k, v = (_rand((1, n, 2, 64), BF, 90 + n) for n in (2, 900, 900))
    out = torch.empty_like(q)
    F.cross_attention(q, k, v, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.cross_attention(q, k, v, out=out)
    v[0, 40, 1, 3] = INF
    graph.replay()
    torch.cuda.synchronize()
    _check_classes(out, q, k, v)
    v[0, 40, 1, 3] = 1.0
    graph.replay()
    torch.cuda.synchronize()
    _check(out, q, k, v)


@pytest.mark.parametrize("layout", ["heads before tokens", "fused columns", "shared by the batch"])
@pytest.mark.parametrize("D,dtype", [(64, HF), (120, BF)])
def test_infinities_in_views(F, layout, D, dtype):
    # the rows that are made once more are read by plain loads with the tensors' own strides
    B, Lq, Lk, Hq, Hk = 3, 4, 1200, 6, 3
    if layout == "heads before tokens":
        q = _rand((B, Hq, Lq, D + 8), dtype, 140)[..., :D].transpose(1, 2)
        k, v = (_rand((B, Hk, Lk, D + 8), dtype, s)[..., :D].transpose(1, 2) for s in (141, 142))
    elif layout == "fused columns":
        q = _rand((B, Lq, (Hq + 1) * D), dtype, 143)[..., D:].unflatten(2, (Hq, D))
        k, v = _rand((B, Lk, 2, Hk, D), dtype, 144).unbind(2)
    else:
        q = _rand((1, Lq, Hq, D), dtype, 145).expand(B, -1, -1, -1)
        k, v = (_rand((1, Lk, Hk, D), dtype, s).expand(B, -1, -1, -1) for s in (146, 147))
    v[0, 700, 1, D - 1] = INF
    v[-1, 701, 2, 0] = -INF
    lens = torch.tensor([1200, 0, 702], dtype=torch.int32).cuda()
    store = torch.full((B, Lq, Hq, D + 8), 7.0, device="cuda", dtype=dtype)
    F.cross_attention(q, k, v, kv_lens=lens, out=store[..., :D])
    _check_classes(store[..., :D].contiguous(), q, k, v.clone(), lens)
    assert bool((store[..., D:] == 7.0).all()) and bool((store[1, ..., :D] == 0).all())


def test_infinities_on_several_streams_at_once(F):
    sets = [[_rand((2, n, 4, 64), BF, 150 + 10 * i + n) for n in (1, 2000, 2000)] for i in range(4)]
    for i, (_, _, v) in enumerate(sets):
        v[i % 2, 100 * i, i, 2 * i] = INF
    want = [F.cross_attention(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[F.cross_attention(*s, stream=stream) for _ in range(5)] for s, stream in zip(sets, streams)]
    torch.cuda.synchronize()
    for s, w, gs in zip(sets, want, got):
        _check_classes(w, *s)
        assert all(torch.equal(w.view(torch.int16), x.view(torch.int16)) for x in gs)
    F.nvfp4_check_fault()
