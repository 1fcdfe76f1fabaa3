"""GPU parity of rotary positions with several axes against the float64 oracle:
layouts, ladders, norms, strides, far and fractional positions, in place.

Tolerance: one rounding to the type (half a step, eps / 2 of the value, and
half of fp16's smallest subnormal step) plus 2^-17 of |a| + |b|.  The latter
covers the 32-bit part, in units of u = 2^-24, as a relative error of each of
the two terms: the hardware's sine and cosine within 2^-20.9 = 8.6 u, their
argument within 3.2 u rad and its product with 2 pi within 3.2 u, three roundings
of the rotation; a norm's sum of squares passes 8 + 5 additions, so it is within
13 u, half of that after the root, which adds 4 u for rsqrtf, 2 u for the mean
and 2 u for the products: below 64 u = 2^-18 in all.  A position
of 2^31 adds its own 64-bit error, 2^31 * 2^-52 rad = 2^-21, on both sides."""
import numpy as np
import pytest
import torch

from oracle import heads_ref as H
from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    require_gpu()
    import nvfp4_block_scaled_12_b200 as F
    return F


def _check(y, x, positions, axes, what, **kw):
    dtype = y.dtype
    want, scale = H.rope_ref(x.cpu().double().numpy(), positions.cpu().double().numpy(), axes,
                             **{k: v.cpu().double().numpy() if torch.is_tensor(v) else v for k, v in kw.items()})
    tol = np.abs(want) * torch.finfo(dtype).eps / 2 * 1.0001 + 2.0 ** -17 * scale
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = np.abs(y.cpu().double().numpy() - want)
    bad = np.argwhere(~(err <= tol))
    assert bad.size == 0, f"{what}: {len(bad)} of {err.size} off, first {bad[0]}: {err[tuple(bad[0])]}"


def _heads(B, L, H_, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, L, H_, D, generator=g).to(dtype).cuda()


CASES = [  # B, L, Hq, Hk, D, axes, dtype, interleaved, shared, norm
    (1, 1, 1, 1, 8, [8], torch.bfloat16, True, False, False),
    (1, 1, 1, 1, 8, [2, 6], torch.float16, False, False, True),
    (2, 33, 3, 1, 64, [16, 24, 24], torch.bfloat16, False, True, True),
    (2, 33, 3, 1, 64, [16, 24, 24], torch.bfloat16, True, True, False),
    (1, 257, 24, 24, 128, [16, 56, 56], torch.bfloat16, True, False, True),
    (3, 100, 5, 9, 128, [44, 42, 42], torch.float16, False, False, False),
    (1, 50, 17, 2, 72, [8, 8, 18, 30], torch.float16, True, False, True),
    (1, 50, 4, 13, 72, [8, 6, 10], torch.bfloat16, False, False, True),       # 24 of 72 rotate
    (2, 7, 2, 2, 80, [10, 14], torch.bfloat16, True, True, True),
    (1, 19, 8, 3, 96, [48, 48], torch.float16, False, False, True),
    (1, 40, 2, 1, 112, [36, 38, 38], torch.bfloat16, False, False, False),
    (1, 5, 3, 3, 256, [64, 96, 96], torch.bfloat16, False, False, True),
    (1, 5, 3, 3, 256, [256], torch.float16, True, False, True),
    (1, 5000, 9, 10, 64, [20, 22, 22], torch.bfloat16, True, False, True),    # eight heads a unit, a ragged last one
]


@pytest.mark.parametrize("B,L,Hq,Hk,D,axes,dtype,interleaved,shared,norm", CASES)
def test_rope_of_fused_projection_columns(F, B, L, Hq, Hk, D, axes, dtype, interleaved, shared, norm):
    g = torch.Generator().manual_seed(L + D)
    qkv = torch.randn(B, L, (Hq + 2 * Hk) * D, generator=g).to(dtype).cuda()
    before = qkv.clone()
    q = qkv[:, :, :Hq * D].unflatten(2, (Hq, D))
    k = qkv[:, :, Hq * D:(Hq + Hk) * D].unflatten(2, (Hk, D))
    pos = torch.randint(0, 300, (L, len(axes)), generator=g, dtype=torch.int32).cuda()
    wq, wk = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() if norm else None for _ in range(2)]
    yq, yk = F.rope(q, pos, axes, k=k, q_weight=wq, k_weight=wk, interleaved=interleaved, shared=shared)
    assert yq.shape == q.shape and yk.shape == k.shape and yq.dtype == dtype and yq.is_contiguous()
    assert torch.equal(qkv, before)
    for y, x, w, n in ((yq, q, wq, "q"), (yk, k, wk, "k")):
        _check(y, x, pos, axes, n, weight=w, interleaved=interleaved, shared=shared)
    # in place: the Q and K columns change, V stays, the bytes are the same
    F.rope(q, pos, axes, k=k, q_weight=wq, k_weight=wk, interleaved=interleaved, shared=shared, q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(qkv[:, :, (Hq + Hk) * D:], before[:, :, (Hq + Hk) * D:])


@pytest.mark.parametrize("norm_q,norm_k", [(True, False), (False, True)])
def test_norm_of_one_tensor_only(F, norm_q, norm_k):
    q, k = _heads(1, 9, 2, 64, torch.bfloat16, 1), _heads(1, 9, 3, 64, torch.bfloat16, 2)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")[:, None].contiguous()
    w = torch.linspace(0.5, 2, 64).bfloat16().cuda()
    yq, yk = F.rope(q, pos, [64], k=k, q_weight=w if norm_q else None, k_weight=w if norm_k else None, eps=1e-3)
    _check(yq, q, pos, [64], "q", weight=w if norm_q else None, eps=1e-3)
    _check(yk, k, pos, [64], "k", weight=w if norm_k else None, eps=1e-3)


def test_one_tensor_alone_and_another_theta(F):
    q = _heads(2, 31, 4, 128, torch.float16, 3)
    pos = torch.randint(-50, 50, (2, 31, 2), dtype=torch.int32).cuda()   # of each batch entry, some before the origin
    y = F.rope(q, pos, [64, 64], theta=256.0)
    assert torch.is_tensor(y)
    _check(y, q, pos, [64, 64], "q", theta=256.0)


@pytest.mark.parametrize("interleaved", [True, False])
def test_far_and_fractional_positions(F, interleaved):
    q = _heads(1, 64, 2, 64, torch.bfloat16, 4)
    far = torch.stack([torch.arange(64) * 16777213 + 5, 2 ** 31 - 1 - torch.arange(64)], 1).to(torch.int64)
    far = (far % 2 ** 31).to(torch.int32).cuda()
    _check(F.rope(q, far, [32, 32], interleaved=interleaved), q, far, [32, 32], "far", interleaved=interleaved)
    part = (torch.arange(128).view(64, 2).float() * 1234.5678 + 0.1).cuda()
    _check(F.rope(q, part, [32, 32], interleaved=interleaved), q, part, [32, 32], "fractional",
           interleaved=interleaved)


def test_heads_before_tokens_and_padded_outputs(F):
    # a [batch, heads, tokens, width] tensor as a view, an output with padding between its heads
    x = torch.randn(2, 5, 21, 64, device="cuda").bfloat16()
    q = x.transpose(1, 2)
    store = torch.full((2, 21, 5, 80), 7.0, device="cuda", dtype=torch.bfloat16)
    pos = torch.randint(0, 99, (21, 3), dtype=torch.int32).cuda()
    F.rope(q, pos, [16, 16, 16], q_out=store[..., :64])
    _check(store[..., :64], q, pos, [16, 16, 16], "padded")
    assert bool((store[..., 64:] == 7.0).all())


def test_a_broadcast_input(F):
    x = torch.randn(1, 12, 1, 64, device="cuda").bfloat16().expand(3, 12, 4, 64)
    pos = torch.randint(0, 99, (12, 1), dtype=torch.int32).cuda()
    _check(F.rope(x, pos, [64]), x, pos, [64], "broadcast")


def test_graph_replay_and_another_stream(F):
    q = _heads(1, 40, 4, 128, torch.bfloat16, 5)
    pos = torch.randint(0, 99, (40, 3), dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    want = F.rope(q, pos, [16, 56, 56])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = F.rope(q, pos, [16, 56, 56], stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.rope(q, pos, [16, 56, 56], q_out=out)
    pos.add_(3)
    graph.replay()
    torch.cuda.synchronize()
    _check(out, q, pos, [16, 56, 56], "replayed")
    assert not torch.equal(out, want)
