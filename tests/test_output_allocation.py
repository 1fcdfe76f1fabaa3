"""How the helpers allocate outputs on the current stream: by a shortcut past
torch's argument parsing that is none of its public names, so it is used only
where it is there and does what it is expected to, and never under a dispatch
mode, which is to see the allocation."""
import pytest
import torch

import nvfp4_block_scaled_12_b200 as F

GUARDS = "torch._C._dynamo.guards._empty_strided_cuda"


@pytest.fixture
def fresh(monkeypatch):
    """The helpers as they are before their first allocation."""
    monkeypatch.setattr(F, "_torch_module", None)
    monkeypatch.setattr(F, "_direct_empty", None, raising=False)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return monkeypatch


def _another_signature(shape, strides, *, dtype):
    raise AssertionError("never reached")


def _raises(*args):
    raise RuntimeError("not in this build")


def _transposed(shape, strides, dtype):
    return torch.empty_strided(shape[::-1], strides, dtype=dtype)


def _of_another_type(shape, strides, dtype):
    return torch.empty_strided(shape, strides, dtype=torch.float32)


def _elsewhere(shape, strides, dtype):
    return torch.empty_strided(shape, strides, dtype=dtype)  # on the CPU, not on the current device


@pytest.mark.parametrize("shortcut", [_another_signature, _raises, _transposed, _of_another_type, _elsewhere])
@pytest.mark.parametrize("shape", [(7,), (3, 4), (2, 3, 4, 8)])
def test_a_shortcut_that_is_not_what_it_was_is_not_used(fresh, shortcut, shape):
    like = torch.zeros(2, dtype=torch.bfloat16)
    fresh.setattr(GUARDS, shortcut)
    F._torch()  # (what every helper begins with)
    t = F._empty_on(None, shape, like, torch.bfloat16)
    assert t.shape == shape and t.dtype == torch.bfloat16 and t.is_contiguous() and t.device == like.device


def test_without_the_shortcut(fresh):
    fresh.delattr(GUARDS)
    F._torch()
    t = F._empty_on(None, (5, 6), torch.zeros(2), torch.uint8)
    assert t.shape == (5, 6) and t.dtype == torch.uint8


@pytest.mark.gpu
def test_dispatch_modes_see_the_outputs():
    from torch.utils._python_dispatch import TorchDispatchMode
    from tests.gpu_helpers import require_gpu
    require_gpu()

    class Allocated(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.addresses = set()

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if isinstance(out, torch.Tensor):
                self.addresses.add(out.data_ptr())
            return out

    x = torch.randn(3, 128, device="cuda").bfloat16()
    q = torch.randn(1, 4, 2, 64, device="cuda").half()
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    F.quantize_mxfp4(x)
    with Allocated() as mode:
        a = F.quantize_mxfp4(x)
        y = F.gemm_mxfp4(a, F.quantize_mxfp4(torch.randn(64, 128, device="cuda").bfloat16()))
        turned = F.rope(q, pos, [64])
        o = F.cross_attention(turned, q, q)
    assert {a.codes.data_ptr(), a.sf.data_ptr(), y.data_ptr(), turned.data_ptr(), o.data_ptr()} <= mode.addresses


@pytest.mark.gpu
def test_the_shortcut_is_what_the_helpers_take_here():
    from tests.gpu_helpers import require_gpu
    require_gpu()
    for shape in ((7,), (3, 4), (2, 3, 4, 8)):
        t = F._empty_on(None, shape, torch.zeros(1, device="cuda"), torch.float16)
        assert t.shape == shape and t.is_contiguous() and t.is_cuda and t.dtype == torch.float16
    assert F._direct_empty and F._dispatch_modes() == 0
