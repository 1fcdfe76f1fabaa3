"""Pins for the MXFP4 oracle (CPU only): ml_dtypes' element format, blocks that
must round-trip, brute-force nearest search, special blocks, a naive GEMM."""
import ml_dtypes
import numpy as np
import pytest

from oracle import mxfp4_ref as X
from oracle import nvfp4_ref as N

F4 = ml_dtypes.float4_e2m1fn


def test_blocks_scaled_by_one_match_ml_dtypes():
    # a maximum in [4, 8) scales by 2^0: the codes are ml_dtypes' E2M1 of the clamped values
    rng = np.random.default_rng(0)
    x = rng.uniform(-6, 6, (400, 32)).astype(np.float32)
    x[:, 0] = rng.choice([4.0, 5.0, 6.0, 7.5, -4.5], 400)
    codes, sf = X.quantize_mxfp4(x)
    assert np.all(sf == 127)
    want = np.clip(x, -6, 6).astype(F4).view(np.uint8) & 15
    assert np.array_equal(N.unpack_codes(codes), want)


@pytest.mark.parametrize("k", [-100, -3, 0, 5, 100])
def test_representable_blocks_round_trip(k):
    rng = np.random.default_rng(k + 200)
    codes = rng.integers(0, 16, (300, 32)).astype(np.uint8)
    codes[np.arange(300), rng.integers(0, 32, 300)] = rng.choice([6, 7, 14, 15], 300)  # +-4, +-6
    x = N.e2m1_decode(codes).astype(np.float64) * 2.0 ** k
    got, sf = X.quantize_mxfp4(x.astype(np.float32))
    assert np.all(sf == k + 127)
    assert np.array_equal(N.unpack_codes(got), codes)
    assert np.array_equal(X.dequantize_mxfp4(got, sf), x)


def test_block_maximum_scales_into_4_to_8_and_elements_are_nearest():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((200, 64)) * 2.0 ** rng.integers(-30, 30, (200, 1))).astype(np.float32)
    codes, sf = X.quantize_mxfp4(x)
    scale = np.repeat(2.0 ** (sf.astype(np.int64) - 127.0), 32, axis=1)
    top = (np.abs(x) / scale).reshape(200, 2, 32).max(2)
    assert np.all((top >= 4) & (top < 8))
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    best = np.abs(np.abs(x / scale)[..., None] - grid).min(-1)
    got = np.abs(np.abs(x / scale) - np.abs(X.dequantize_mxfp4(codes, sf) / scale))
    assert np.array_equal(got, best)


def test_special_blocks():
    x = np.zeros((4, 32), np.float32)
    x[0, 3] = -0.0
    x[1, 5] = 2.0 ** -133            # the smallest bf16 value
    x[2, :] = 3.3e38                 # near bf16's largest
    x[3, :2] = [7.75, -0.25]         # saturates to 6; ties to the even code 0, sign kept
    codes, sf = X.quantize_mxfp4(x)
    q = N.unpack_codes(codes)
    assert list(sf[:, 0]) == [0, 0, 252, 127]
    assert q[0, 3] == 8 and np.count_nonzero(q[0]) == 1
    assert q[1, 5] == 0              # 2^-133 / 2^-127 = 2^-6, below half of 0.5
    assert np.all(q[2] == 7)         # 3.3e38 / 2^125 = 7.76: clamped to 6, code 7
    q3 = q[3, :2]
    assert list(q3) == [7, 8]
    x = np.full((1, 32), 2.0 ** -126, np.float32)   # exponent -128, clamped to -127: 2^-126 / 2^-127 = 2
    codes, sf = X.quantize_mxfp4(x)
    assert sf[0, 0] == 0 and np.all(N.unpack_codes(codes) == 4)


def test_gemm_and_tolerance_against_a_naive_sum():
    rng = np.random.default_rng(4)
    a_c, a_s = X.quantize_mxfp4(rng.standard_normal((3, 64)).astype(np.float32))
    b_c, b_s = X.quantize_mxfp4(rng.standard_normal((5, 64)).astype(np.float32))
    bias = rng.standard_normal(5)
    y = X.gemm_ref_mxfp4(a_c, a_s, b_c, b_s, alpha=0.5, bias=bias)
    a, b = X.dequantize_mxfp4(a_c, a_s), X.dequantize_mxfp4(b_c, b_s)
    for m in range(3):
        for n in range(5):
            assert abs(y[m, n] - (0.5 * sum(a[m, k] * b[n, k] for k in range(64)) + bias[n])) < 1e-9
    # the bound admits an fp32 sum in another order and refuses a dropped block or a doubled scale
    tol = X.gemm_tolerance_mxfp4(a_c, a_s, b_c, b_s, y, alpha=0.5)
    f = np.float32(0.5) * (a.astype(np.float32)[:, ::-1] @ b.astype(np.float32)[:, ::-1].T) + bias.astype(np.float32)
    assert np.all(np.abs(f - y) <= tol)
    dropped = 0.5 * (a[:, :32] @ b[:, :32].T) + bias
    assert np.any(np.abs(dropped - y) > tol)
    doubled = a.copy()
    doubled[:, 32:] *= 2
    assert np.any(np.abs(0.5 * (doubled @ b.T) + bias - y) > tol)
