"""Argument checks of the MXFP4 entry points, on the CPU: the C ABI refuses
before it touches a device, the torch helpers before they hand a pointer on."""
import pytest
import torch

import nvfp4_block_scaled_12_b200 as F
from tests.test_abi import P, _expect
from tests.test_binding_checks import empty


@pytest.mark.parametrize("rows,k,want", [(4608, 12288, 4608 * 384), (1, 64, 512), (129, 160, 256 * 8), (0, 64, 0),
                                         (5, 16, 0), (5, 48, 0)])
def test_sf_bytes(rows, k, want):
    assert F.nvfp4_mxfp4_sf_bytes(rows, k) == want
    if want:
        assert F._mxfp4_sf_bytes(rows, k) == want


def test_entry_points_reject_bad_arguments():
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_quantize, 0, 16, 64, P, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_quantize, P, 0, 64, P, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_quantize, P, 4, 96, P, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_quantize, P, 1 << 30, 64, P, P, 0)
    _expect(F.NVFP4_EALIGN, F.nvfp4_mxfp4_quantize, P, 4, 64, P + 8, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_gemm, P, P, P, P, 0, 64, 64, 1.0, 0, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_gemm, P, P, P, P, 16, 12, 64, 1.0, 0, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_gemm, P, P, P, P, 16, 64, 96, 1.0, 0, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_gemm, P, P, P, P, 16, 64, 64, float("nan"), 0, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_gemm, P, P, 0, P, 16, 64, 64, 1.0, 0, P, 0)
    _expect(F.NVFP4_EINVAL, F.nvfp4_mxfp4_gemm, P, P, P, P, 16, 64, 64, 1.0, 0, 0, 0)
    _expect(F.NVFP4_EALIGN, F.nvfp4_mxfp4_gemm, P, P, P, P, 16, 64, 64, 1.0, P + 2, P, 0)


@pytest.fixture
def calls(monkeypatch):
    rec = []
    for name in ("nvfp4_mxfp4_quantize", "nvfp4_mxfp4_gemm"):
        monkeypatch.setattr(F, name, lambda *a, _n=name: rec.append(_n))
    monkeypatch.setattr(F, "_stream", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return rec


def mxfp4(rows, k, dev=0):
    return F.MXFP4Tensor(empty(rows, k // 2, dev=dev), empty(F.nvfp4_mxfp4_sf_bytes(rows, k), dev=dev), rows, k)


def test_helpers_pass_well_formed_buffers_and_refuse_others(calls):
    bf = torch.bfloat16
    M, N, K = 130, 192, 320
    x, a, b, y = empty(M, K, dtype=bf), mxfp4(M, K), mxfp4(N, K), empty(M, N, dtype=bf)
    F.quantize_mxfp4(x, out=a)
    F.gemm_mxfp4(a, b, bias=empty(N, dtype=bf), y=y)
    assert calls == ["nvfp4_mxfp4_quantize", "nvfp4_mxfp4_gemm"]
    small = F.MXFP4Tensor(a.codes, empty(F.nvfp4_mxfp4_sf_bytes(M, K) - 1), M, K)
    for bad in (lambda: F.quantize_mxfp4(empty(M, K, dtype=torch.float16), out=a),
                lambda: F.quantize_mxfp4(empty(K, M, dtype=bf).t(), out=a),
                lambda: F.quantize_mxfp4(empty(M, K, dtype=bf, dev=1), out=a),
                lambda: F.quantize_mxfp4(x, out=small),
                lambda: F.quantize_mxfp4(x, out=mxfp4(M, 2 * K)),
                lambda: F.gemm_mxfp4(a, mxfp4(N, 2 * K), y=y),
                lambda: F.gemm_mxfp4(small, b, y=y),
                lambda: F.gemm_mxfp4(a, b, y=empty(M, N + 8, dtype=bf)),
                lambda: F.gemm_mxfp4(a, b, y=empty(M, N, dtype=torch.float16)),
                lambda: F.gemm_mxfp4(a, b, bias=empty(N + 1, dtype=bf), y=y),
                lambda: F.gemm_mxfp4(a, mxfp4(N, K, dev=1), y=y)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    assert len(calls) == 2
