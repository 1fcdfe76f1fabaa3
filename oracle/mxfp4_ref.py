"""Plain CPU oracle for the MXFP4 variant of the linear-layer hot path.

TEST INFRASTRUCTURE ONLY (same rules as ``oracle/nvfp4_ref.py``): only
``tests/`` uses it, and it imports nothing from the CUDA library.

MXFP4 is the 4-bit format of the Open Compute Project microscaling standard:
E2M1 elements in 32-element blocks that share one power-of-two scale (E8M0).
The conversion is MXFP8's with E2M1's constants: ``X = 2^(floor(log2(max_i
|V_i|)) - 2)`` (2 is the exponent of E2M1's largest normal, 6 = 1.5 * 2^2),
``P_i = V_i / X`` rounded to nearest, ties to the even code, clamped at 6.

The choices that the standard leaves open are MXFP8's (``oracle/mxfp8_ref.py``):
an all-zero block has scale byte 0 and zeros that keep their sign, the shared
exponent is clamped into [-127, 127], and the division is the fp32 product
``V_i * 2^-s``.

Pins: tests/test_oracle_mxfp4.py (element codes vs ml_dtypes float4_e2m1fn,
blocks of representable values round-trip, the block maximum scales into
[4, 8), brute-force nearest element, zero and saturating blocks, brute-force
GEMM).
"""
from __future__ import annotations

import numpy as np

from .mxfp8_ref import (MX_BLOCK, block_exponent, e8m0_decode, sf_bytes_mxfp8, swizzle_sf_mxfp8,
                        unswizzle_sf_mxfp8)
from .nvfp4_ref import e2m1_decode, e2m1_encode, pack_codes, unpack_codes

#: Exponent of E2M1's largest normal value (6 = 1.5 * 2^2).
E2M1_EMAX = 2

# the scale buffer is MXFP8's
sf_bytes_mxfp4, swizzle_sf_mxfp4, unswizzle_sf_mxfp4 = sf_bytes_mxfp8, swizzle_sf_mxfp8, unswizzle_sf_mxfp8


def quantize_mxfp4(x):
    """Quantize ``x`` [rows, K] (fp32-exact values, e.g. bf16 inputs) to MXFP4.

    Returns ``(codes, sf)``: ``codes`` uint8 [rows, K/2], two E2M1 codes to a
    byte; ``sf`` uint8 [rows, K/32], the E8M0 block scales row-major.
    """
    x = np.asarray(x, dtype=np.float32)
    rows, K = x.shape
    if K % MX_BLOCK:
        raise ValueError("K must be a multiple of 32")
    blocks = x.reshape(rows, K // MX_BLOCK, MX_BLOCK)
    amax = np.max(np.abs(blocks), axis=2).astype(np.float64)
    e = np.where(amax > 0, block_exponent(np.where(amax > 0, amax, 1.0)), 0)
    s = np.where(amax > 0, np.clip(e - E2M1_EMAX, -127, 127), -127)
    inv = np.ldexp(np.float32(1.0), -s).astype(np.float32)           # 2^-s, exact in fp32
    scaled = (blocks * inv[:, :, None]).astype(np.float32)            # one fp32 multiply
    codes = e2m1_encode(scaled).reshape(rows, K)
    return pack_codes(codes), (s + 127).astype(np.uint8)


def dequantize_mxfp4(codes, sf) -> np.ndarray:
    """x_hat = e2m1(code) * 2^(scale - 127), float64 [rows, K]."""
    vals = np.asarray(e2m1_decode(unpack_codes(codes)), dtype=np.float64)
    rows, K = vals.shape
    return (vals.reshape(rows, K // MX_BLOCK, MX_BLOCK) * e8m0_decode(sf)[:, :, None]).reshape(rows, K)


def gemm_ref_mxfp4(a_codes, a_sf, b_codes, b_sf, alpha=1.0, bias=None) -> np.ndarray:
    """``y = alpha * a_hat @ b_hat^T + bias`` in float64."""
    y = np.float64(np.float32(alpha)) * (dequantize_mxfp4(a_codes, a_sf) @ dequantize_mxfp4(b_codes, b_sf).T)
    return y if bias is None else y + np.asarray(bias, dtype=np.float64)[None, :]


def gemm_tolerance_mxfp4(a_codes, a_sf, b_codes, b_sf, y_ref, alpha=1.0) -> np.ndarray:
    """Bound of an fp32 sum of K exact products in any order, the fma that adds
    the bias, and one bf16 rounding: every product of E2M1 values and powers of
    two is exact, so |error| <= K * 2^-23 * sum_k |a_k b_k| (Higham, Accuracy
    and Stability, section 3.1, with one unit 2^-23 per addition, which also
    admits a truncating adder), times 1.01 for its own rounding, plus 2^-8 |y|
    for the bf16 rounding (half a step is at most 2^-8 of the value) with a
    thousandth of it for the fma's."""
    a, b = np.abs(dequantize_mxfp4(a_codes, a_sf)), np.abs(dequantize_mxfp4(b_codes, b_sf))
    return abs(float(np.float32(alpha))) * 1.01 * a.shape[1] * 2.0 ** -23 * (a @ b.T) + 2.0 ** -8 * np.abs(y_ref) * 1.001


__all__ = ["MX_BLOCK", "E2M1_EMAX", "quantize_mxfp4", "dequantize_mxfp4", "sf_bytes_mxfp4", "swizzle_sf_mxfp4",
           "unswizzle_sf_mxfp4", "gemm_ref_mxfp4", "gemm_tolerance_mxfp4"]
