"""Rotary positions on shapes whose units (the lanes that share their sines and
cosines) take several heads each: heads that step from one to the next, loads
ahead of them, and tensors cut into units of which the last is shorter.  The
tolerance is the rotary tests'; the plan is asked on the host for the present
device, so that the cases stay what they are written for."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_rope import _check

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


CASES = [  # B, L, Hq, Hk, D, axes, units (of q, of k), heads of a unit (of q, of k)
    (1, 1300, 25, 29, 128, [16, 56, 56], (2, 2), (13, 15)),   # a last unit of 12, and of 14 heads
    (2, 1600, 9, 25, 64, [8, 16, 16], (1, 2), (9, 13)),       # 24 of 64 elements pass through
    (1, 3000, 6, 5, 256, [64, 96, 96], (1, 1), (6, 5)),
    (3, 700, 14, 1, 72, [8, 8, 18, 30], (2, 1), (7, 1)),      # nine of sixteen lanes at work
]


@pytest.mark.parametrize("B,L,Hq,Hk,D,axes,units,heads", CASES)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_units_of_several_heads(F, B, L, Hq, Hk, D, axes, units, heads, dtype, interleaved, norm):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert F.nvfp4_rope_plan(Hq, Hk, B * L, D, sms) == (*heads, *units)
    g = torch.Generator().manual_seed(L + D)
    qkv = torch.randn(B, L, (Hq + Hk + 1) * D, generator=g).to(dtype).cuda()
    before = qkv.clone()
    q = qkv[:, :, :Hq * D].unflatten(2, (Hq, D))
    k = qkv[:, :, Hq * D:(Hq + Hk) * D].unflatten(2, (Hk, D))
    pos = torch.randint(0, 300, (B, L, len(axes)), generator=g, dtype=torch.int32).cuda()
    wq, wk = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() if norm else None for _ in range(2)]
    yq, yk = F.rope(q, pos, axes, k=k, q_weight=wq, k_weight=wk, interleaved=interleaved)
    assert torch.equal(qkv, before)
    for y, x, w, n in ((yq, q, wq, "q"), (yk, k, wk, "k")):
        _check(y, x, pos, axes, n, weight=w, interleaved=interleaved)
    # in place: the Q and K columns change, what follows them stays, the bytes are the same
    F.rope(q, pos, axes, k=k, q_weight=wq, k_weight=wk, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(qkv[:, :, (Hq + Hk) * D:], before[:, :, (Hq + Hk) * D:])


@pytest.mark.parametrize("norm_q,norm_k", [(True, False), (False, True)])
def test_one_tensor_normed_in_units_of_several_heads(F, norm_q, norm_k):
    g = torch.Generator().manual_seed(5)
    q, k = (torch.randn(1, 1400, h, 128, generator=g).to(BF).cuda() for h in (26, 3))
    pos = torch.randint(0, 300, (1400, 1), generator=g, dtype=torch.int32).cuda()
    w = torch.linspace(0.5, 2, 128).to(BF).cuda()
    weights = dict(q_weight=w if norm_q else None, k_weight=w if norm_k else None)
    # (an output with padding between its heads: each steps by its own stride)
    store = torch.full((1, 1400, 26, 136), 7.0, device="cuda", dtype=BF)
    yq, yk = F.rope(q, pos, [128], k=k, q_out=store[..., :128], **weights)
    _check(yq, q, pos, [128], "q", weight=weights["q_weight"])
    _check(yk, k, pos, [128], "k", weight=weights["k_weight"])
    assert bool((store[..., 128:] == 7.0).all())
