"""Argument checks of the entry points on 16-bit heads, on the CPU: the C ABI
refuses before it touches a device, the torch helpers before they hand a
pointer on."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_12_b200 as F
from tests.test_abi import P, _expect
from tests.test_binding_checks import empty

BF = torch.bfloat16
Q, R = P + (1 << 24), P + (2 << 24)


def heads(batch=64 * 512, token=512, head=64, data=P):
    return F.Heads(data, batch, token, head)


def rope_args(**kw):
    a = dict(tensors=[F.RopeTensor(heads(), heads(), 8, 0)], batch=2, tokens=64, head_dim=64, dtype=0, positions=P,
             pos_type=0, pos_batch_stride=0, axis_dims=[16, 24, 24], theta=1e4, flags=1, eps=1e-6, stream=0)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(tensors=[]), dict(batch=0), dict(tokens=0), dict(batch=1 << 20, tokens=1 << 20), dict(head_dim=60),
    dict(head_dim=264), dict(head_dim=0), dict(dtype=2), dict(positions=0), dict(pos_type=2),
    dict(pos_batch_stride=-1), dict(axis_dims=[]), dict(axis_dims=[8] * 5), dict(axis_dims=[15, 25]),
    dict(axis_dims=[64, 2]), dict(axis_dims=[10, 10]), dict(axis_dims=[0, 8]), dict(theta=0.0),
    dict(theta=float("nan")), dict(theta=float("inf")), dict(flags=4), dict(eps=-1.0), dict(eps=float("nan")),
    dict(tensors=[F.RopeTensor(heads(), heads(), 0, 0)]), dict(tensors=[F.RopeTensor(heads(), heads(), 1 << 20, 0)]),
    dict(tensors=[F.RopeTensor(heads(data=0), heads(), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(token=508), heads(), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(token=-512), heads(), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(head=56, data=Q), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(batch=0, data=Q), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(), 8, 0)] * 3),
    # outputs that overlap themselves: tokens inside one another's heads, batches inside one another's tokens
    dict(tensors=[F.RopeTensor(heads(), heads(token=64, data=Q), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(batch=63 * 512, data=Q), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(token=64, head=128, data=Q), 8, 0)]),
    # in place with other strides; the second tensor's output as the first's, its input as the first's output
    dict(tensors=[F.RopeTensor(heads(), heads(token=64, head=64 * 64), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(data=Q), 8, 0), F.RopeTensor(heads(data=R), heads(data=Q), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(data=Q), 8, 0), F.RopeTensor(heads(data=Q), heads(data=R), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(data=Q), 8, 0), F.RopeTensor(heads(data=R), heads(), 8, 0)])])
def test_rope_rejects_bad_arguments(kw):
    _expect(F.NVFP4_EINVAL, F.nvfp4_rope, *rope_args(**kw))


@pytest.mark.parametrize("kw", [
    dict(positions=P + 2), dict(tensors=[F.RopeTensor(heads(data=P + 8), heads(), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(data=P + 2), 8, 0)]),
    dict(tensors=[F.RopeTensor(heads(), heads(), 8, P + 4)])])
def test_rope_rejects_unaligned_pointers(kw):
    _expect(F.NVFP4_EALIGN, F.nvfp4_rope, *rope_args(**kw))


@pytest.fixture
def calls(monkeypatch):
    rec = []
    for name in ("nvfp4_rope", "nvfp4_attention"):
        monkeypatch.setattr(F, name, lambda *a, _n=name: rec.append((_n, a)))
    monkeypatch.setattr(F, "_stream", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return rec


def test_rope_helper(calls):
    q, k = empty(2, 9, 4, 64, dtype=BF), empty(2, 9, 2, 64, dtype=BF)
    qo, ko = empty(2, 9, 4, 64, dtype=BF), empty(2, 9, 2, 64, dtype=BF)
    pos, w = empty(9, 2, dtype=torch.int32), empty(64, dtype=BF)
    got = F.rope(q, pos, [32, 32], k=k, q_weight=w, q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko
    assert F.rope(q, empty(2, 9, 2, dtype=torch.float32), [32, 32], q_out=q) is q
    (_, a), (_, b) = calls
    first, second = (F.RopeTensor.from_buffer_copy(a[0], i * len(a[0]) // 2) for i in range(2))
    assert len(a[0]) == 2 * ctypes.sizeof(F.RopeTensor) and first.norm_weight and not second.norm_weight
    assert (first.heads, second.heads) == (4, 2) and first.in_.data == q.data_ptr() and second.out.data == ko.data_ptr()
    assert (first.in_.batch_stride, first.in_.token_stride, first.in_.head_stride) == (9 * 256, 256, 64)
    assert a[1:5] == (2, 9, 64, 0) and a[6] == F.POS_INT32 and a[7] == 0 and b[6] == F.POS_FLOAT32 and b[7] == 18
    wide = empty(2, 9, 4, 128, dtype=BF)
    for bad in (lambda: F.rope(empty(2, 9, 4, 64, dtype=torch.float32), pos, [32, 32], q_out=qo),
                lambda: F.rope(q[0], pos, [32, 32], q_out=qo),
                lambda: F.rope(wide[..., ::2], pos, [32, 32], q_out=qo),
                lambda: F.rope(empty(2, 9, 4, 64, dtype=BF, dev=1), pos, [32, 32], q_out=qo),
                lambda: F.rope(q, pos, [32, 32], q_out=ko),
                lambda: F.rope(q, pos, [32, 32], q_out=empty(2, 9, 4, 64, dtype=torch.float16)),
                lambda: F.rope(q, pos, [32, 32], k=empty(2, 8, 2, 64, dtype=BF), q_out=qo, k_out=ko),
                lambda: F.rope(q, pos, [32, 32], k=empty(2, 9, 2, 72, dtype=BF), q_out=qo),
                lambda: F.rope(q, pos, [32, 32], k=empty(2, 9, 2, 64, dtype=torch.float16), q_out=qo),
                lambda: F.rope(q, pos, [32, 32], k_weight=w, q_out=qo),
                lambda: F.rope(q, pos, [32, 32], q_weight=empty(32, dtype=BF), q_out=qo),
                lambda: F.rope(q, pos, [32, 32], q_weight=empty(64, dtype=torch.float32), q_out=qo),
                lambda: F.rope(q, pos, [64], q_out=qo),
                lambda: F.rope(q, empty(8, 2, dtype=torch.int32), [32, 32], q_out=qo),
                lambda: F.rope(q, empty(9, 2, dtype=torch.int64), [32, 32], q_out=qo),
                lambda: F.rope(q, empty(9, 2, dtype=torch.int32, dev=1), [32, 32], q_out=qo),
                lambda: F.rope(q, empty(2, 9, dtype=torch.int32).t(), [32, 32], q_out=qo),
                lambda: F.rope(empty(2, 0, 4, 64, dtype=BF), empty(0, 2, dtype=torch.int32), [32, 32])):
        with pytest.raises((TypeError, ValueError)):
            bad()
    assert len(calls) == 2


def attention_args(**kw):
    a = dict(q=heads(), k=heads(), v=heads(), out=heads(data=Q), batch=2, q_tokens=64, kv_tokens=64, q_heads=8, kv_heads=8,
             head_dim=64, dtype=0, kv_lens=0, scale=0.125, stream=0)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(q_tokens=0), dict(kv_tokens=0), dict(q_heads=0), dict(kv_heads=0), dict(head_dim=0),
    dict(head_dim=68), dict(head_dim=136), dict(q_heads=8, kv_heads=3), dict(q_heads=258, kv_heads=2, batch=1),
    dict(dtype=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(scale=3e38), dict(batch=1 << 29, kv_heads=8), dict(q=heads(data=0)), dict(out=heads(data=0)), dict(k=heads(token=4)),
    dict(v=heads(head=-64)), dict(k=heads(token=0)), dict(q=heads(head=0)), dict(out=heads(batch=0, data=Q)),
    dict(out=heads(head=56, data=Q)), dict(k=heads(batch=1 << 40)), dict(out=heads()), dict(q=heads(data=Q)),
    dict(v=heads(data=Q)), dict(out=heads(token=64, data=Q)), dict(out=heads(batch=63 * 512, data=Q))])
def test_attention_rejects_bad_arguments(kw):
    _expect(F.NVFP4_EINVAL, F.nvfp4_attention, *attention_args(**kw))


@pytest.mark.parametrize("kw", [dict(q=heads(data=P + 8)), dict(v=heads(data=P + 2)), dict(out=heads(data=P + 8)),
                                dict(kv_lens=P + 2)])
def test_attention_rejects_unaligned_pointers(kw):
    _expect(F.NVFP4_EALIGN, F.nvfp4_attention, *attention_args(**kw))


def test_attention_helper(calls):
    q, k, v, out = (empty(2, n, h, 64, dtype=BF) for n, h in ((9, 4), (33, 2), (33, 2), (9, 4)))
    lens = empty(2, dtype=torch.int32)
    assert F.cross_attention(q, k, v, kv_lens=lens, out=out) is out
    F.cross_attention(q, k, v, scale=0.3, out=out)
    (_, a), (_, b) = calls
    assert a[4:11] == (2, 9, 33, 4, 2, 64, 0) and a[11] and abs(a[12] - 0.125) < 1e-12
    assert b[11] == 0 and b[12] == 0.3
    h16 = torch.float16
    for bad in (lambda: F.cross_attention(q, k, empty(2, 32, 2, 64, dtype=BF), out=out),
                lambda: F.cross_attention(q, k, empty(2, 33, 2, 64, dtype=h16), out=out),
                lambda: F.cross_attention(q, empty(3, 33, 2, 64, dtype=BF), empty(3, 33, 2, 64, dtype=BF), out=out),
                lambda: F.cross_attention(q, empty(2, 33, 2, 72, dtype=BF), empty(2, 33, 2, 72, dtype=BF), out=out),
                lambda: F.cross_attention(empty(2, 9, 4, 64, dtype=torch.float32), k, v, out=out),
                lambda: F.cross_attention(q, k, v, kv_lens=empty(3, dtype=torch.int32), out=out),
                lambda: F.cross_attention(q, k, v, kv_lens=empty(2, dtype=torch.int64), out=out),
                lambda: F.cross_attention(q, k, v, kv_lens=empty(2, dtype=torch.int32, dev=1), out=out),
                lambda: F.cross_attention(q, k, v, out=empty(2, 9, 2, 64, dtype=BF)),
                lambda: F.cross_attention(q, empty(2, 33, 2, 64, dtype=BF, dev=1), v, out=out),
                lambda: F.cross_attention(q, empty(2, 0, 2, 64, dtype=BF), empty(2, 0, 2, 64, dtype=BF), out=out),
                lambda: F.cross_attention(q.transpose(2, 3), k, v, out=out)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    assert len(calls) == 2


@pytest.mark.parametrize("out", [heads(data=Q), heads(token=64, head=64 * 64, data=Q),  # [batch, heads, tokens, width]
                                 heads(batch=512, token=2 * 512, data=Q),                # [tokens, batch, heads, width]
                                 heads(batch=64 * 1536, token=1536, data=Q)])            # columns of a wider buffer
def test_outputs_of_any_order_pass_the_checks(out):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU: the pointers are not real")
    for call in (lambda: F.nvfp4_attention(*attention_args(out=out)),
                 lambda: F.nvfp4_rope(*rope_args(tensors=[F.RopeTensor(heads(), out, 8, 0)])),
                 lambda: F.nvfp4_rope(*rope_args(tensors=[F.RopeTensor(out, out, 8, 0)]))):
        with pytest.raises(F.NVFP4Error) as e:  # (no device to run on: that, not the arguments, ends the call)
            call()
        assert e.value.status in (F.NVFP4_ECUDA, F.NVFP4_EARCH)
