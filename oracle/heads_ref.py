"""Plain CPU oracle for what runs on 16-bit heads between the linear layers:
rotary positions with several axes, and attention over states of another
length, both in float64.

TEST INFRASTRUCTURE ONLY (same rules as ``oracle/nvfp4_ref.py``).

Pins: tests/test_oracle_heads.py (rotations against complex numbers, against
their defining property that the product of two rotated heads depends on the
difference of the positions alone; attention against a loop over queries).
"""
from __future__ import annotations

import numpy as np


def rope_angles(positions, axes, theta=10000.0, shared=False) -> np.ndarray:
    """Angle of every position and pair, [..., R/2], in float64."""
    positions = np.asarray(positions, dtype=np.float64)
    total, out, at = sum(axes), [], 0
    for a, width in enumerate(axes):
        i = np.arange(width // 2)
        f = theta ** (-2.0 * (at + i) / total) if shared else theta ** (-2.0 * i / width)
        out.append(positions[..., a:a + 1] * f)
        at += width // 2
    return np.concatenate(out, axis=-1)


def rope_ref(x, positions, axes, theta=10000.0, weight=None, eps=1e-6, interleaved=True, shared=False):
    """``(y, scale)`` for ``x`` [B, L, H, D] and ``positions`` [L, A] or [B, L, A]:
    the rotated heads and, per element, |a| + |b| of its pair (|x| where it
    passes through), which bounds what a relative error of the sines, cosines
    and the norm can change."""
    x = np.asarray(x, dtype=np.float64)
    total = sum(axes)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    angle = rope_angles(positions, axes, theta, shared)[..., :, None, :]  # [.., L, 1, R/2]
    c, s = np.cos(angle), np.sin(angle)
    if interleaved:
        ia, ib = np.arange(0, total, 2), np.arange(1, total, 2)
    else:
        ia, ib = np.arange(total // 2), np.arange(total // 2, total)
    y, scale = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    scale[..., ia] = scale[..., ib] = np.abs(a) + np.abs(b)
    return y, scale


def attention_ref(q, k, v, kv_lens=None, scale=None):
    """``(o, weight)`` for q [B, Lq, Hq, D], k and v [B, Lk, Hk, D]: per head
    softmax(scale q k^T) v over the first kv_lens[b] keys (zeros where there is
    none), and the same with |v|: what a relative error of every probability
    can change."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    B, _, Hq, D = q.shape
    group = Hq // k.shape[2]
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    o, w = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = k.shape[1] if kv_lens is None else int(np.clip(kv_lens[b], 0, k.shape[1]))
        if n == 0:
            continue
        for h in range(Hq):
            kk, vv = k[b, :n, h // group], v[b, :n, h // group]
            s = scale * (q[b, :, h] @ kk.T)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o[b, :, h], w[b, :, h] = p @ vv, p @ np.abs(vv)
    return o, w


__all__ = ["rope_angles", "rope_ref", "attention_ref"]
