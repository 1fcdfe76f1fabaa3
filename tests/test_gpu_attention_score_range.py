"""Scores whose product with the scale leaves the range of fp32.  They count as
the infinity that fp32 makes of them: +inf gives its row NaN (inf - inf), -inf
a probability of zero, and a row that has nothing else zeros, as scores that
are -inf by themselves do."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_attention import BF, HF, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


# few rows over split keys, whole tiles joined, whole items in turn
@pytest.mark.parametrize("Lq,Lk", [(2, 1500), (200, 1500), (3000, 300)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_whose_scores_all_overflow(F, Lq, Lk, dtype, sign):
    q = torch.zeros(1, Lq, 2, 64, device="cuda", dtype=dtype)
    k = torch.ones(1, Lk, 2, 64, device="cuda", dtype=dtype)
    v = _rand((1, Lk, 2, 64), dtype, 1)
    q[:, ::2] = sign     # every score of these rows is +-64, scaled +-64e37
    o = F.cross_attention(q, k, v, scale=1e37)
    assert bool((torch.isnan(o[:, ::2]) if sign > 0 else o[:, ::2] == 0).all())
    assert bool(torch.isfinite(o[:, 1::2]).all())


@pytest.mark.parametrize("Lq,Lk", [(2, 1500), (200, 1500), (3000, 300)])
def test_the_overflow_may_come_in_a_later_tile(F, Lq, Lk):
    q = torch.zeros(1, Lq, 2, 64, device="cuda", dtype=BF)
    q[:, ::2] = 1.0
    k = torch.zeros(1, Lk, 2, 64, device="cuda", dtype=BF)
    k[:, Lk - 20:] = 1.0
    o = F.cross_attention(q, k, _rand((1, Lk, 2, 64), BF, 2), scale=1e37)
    assert bool(torch.isnan(o[:, ::2]).all())
    assert bool(torch.isfinite(o[:, 1::2]).all())


@pytest.mark.parametrize("Lq,Lk", [(2, 1500), (200, 1500), (3000, 300)])
@pytest.mark.parametrize("at", [5, 200, -1])
def test_an_overflow_far_below_the_largest_score_is_a_probability_of_zero(F, Lq, Lk, at):
    # one key scores 0, all others -64 (scaled -64e37): tiles, and parts of shared keys, with nothing but those
    q = torch.ones(1, Lq, 2, 64, device="cuda", dtype=BF)
    k = -torch.ones(1, Lk, 2, 64, device="cuda", dtype=BF)
    at %= Lk
    k[:, at] = 0.0
    v = _rand((1, Lk, 2, 64), BF, 3)
    o = F.cross_attention(q, k, v, scale=1e37)
    assert torch.equal(o, v[:, at:at + 1].expand_as(o))
