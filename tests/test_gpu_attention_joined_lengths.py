"""Attention whose queries fill more than 32 rows a K/V head while its items
are too few for the device: whole query tiles, one (its two slots take the key
tiles in turn) or two, with the keys split over a cluster of up to 8 CTAs and
joined.  Each batch entry has its own length, with rubbish behind it: lengths
that leave ranks, or slots, without a key tile, that end inside a rank's last
tile or on its edge, and none at all.  The tolerance is the attention tests'.

That these shapes are split follows from the launch's cost in key tiles: 12
tiles of 1500 states against ceil(12 / 8) + 3 = 5 for clusters of eight, of
which 16 to 18 fit, with 8 and 6 items; 40 tiles against 8 of 5000."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_attention import BF, HF, _check, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


LENGTHS = [  # of four entries each
    [0, 1, 129, 1499],
    [1500, 128, 127, 0],
    [16, 255, 256, 257],
    [1000, 1024, 1025, 1039],
]


@pytest.mark.parametrize("Lq", [60, 128, 200, 256])
@pytest.mark.parametrize("D,dtype", [(64, HF), (72, BF), (128, BF), (128, HF)])
@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("rubbish", [float("nan"), float("inf")])
def test_lengths_of_joined_items(F, Lq, D, dtype, lens, rubbish):
    q, k, v = (_rand((4, n, 2, D), dtype, 100 + n + i) for i, n in enumerate((Lq, 1500, 1500)))
    for b, n in enumerate(lens):
        k[b, n:] = rubbish
        v[b, n:] = rubbish
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    o = F.cross_attention(q, k, v, kv_lens=n)
    _check(o, q, k, v, n)
    for b, m in enumerate(lens):
        if m == 0:
            assert bool((o[b] == 0).all())
    assert torch.equal(o, F.cross_attention(q, k, v, kv_lens=n))


@pytest.mark.parametrize("Lq,Hq,Hk,D,dtype", [(50, 6, 3, 96, BF), (17, 10, 2, 128, HF), (100, 2, 1, 40, BF)])
def test_lengths_of_joined_items_with_shared_heads(F, Lq, Hq, Hk, D, dtype):
    # groups that do not divide a tile, rows of the tile without a query, entries on both sides of a rank's edge
    lens = [4999, 0, 641, 640, 639, 5000]
    q, k, v = _rand((6, Lq, Hq, D), dtype, 120), _rand((6, 5000, Hk, D), dtype, 121), _rand((6, 5000, Hk, D), dtype, 122)
    for b, n in enumerate(lens):
        k[b, n:] = float("-inf")
        v[b, n:] = float("nan")
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    store = torch.full((6, Lq + 2, Hq, D + 8), 7.0, device="cuda", dtype=dtype)
    out = store[:, 1:-1, :, :D]
    F.cross_attention(q, k, v, kv_lens=n, out=out)
    _check(out, q, k, v, n)
    assert bool((store[:, [0, -1]] == 7.0).all()) and bool((store[..., D:] == 7.0).all())


def test_lengths_clamped_and_changed_under_a_replay(F):
    q, k, v = (_rand((4, n, 2, 128), BF, 130 + n) for n in (150, 1500, 1500))
    n = torch.tensor([1500, 700, 2 ** 31 - 1, -9], dtype=torch.int32).cuda()
    out = F.cross_attention(q, k, v, kv_lens=n)
    _check(out, q, k, v, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.cross_attention(q, k, v, kv_lens=n, out=out)
    for lens in ([1, 0, 1500, 130], [-(2 ** 31), 1499, 3, 640]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        _check(out, q, k, v, n)


def test_no_kernel_reported_a_fault(F):
    torch.cuda.synchronize()
    F.nvfp4_check_fault()
