"""Pins for the oracle of rotary positions and attention (CPU only)."""
import numpy as np
import pytest

from oracle import heads_ref as H


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("shared", [True, False])
def test_rotated_products_depend_on_the_difference_of_positions(interleaved, shared):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((1, 1, 1, 24)), rng.standard_normal((1, 1, 1, 24))
    axes = [4, 8, 4]
    pq, pk, shift = rng.integers(0, 50, (1, 3)), rng.integers(0, 50, (1, 3)), rng.integers(0, 1000, (1, 3))

    def product(p1, p2):
        a, _ = H.rope_ref(q, p1, axes, interleaved=interleaved, shared=shared)
        b, _ = H.rope_ref(k, p2, axes, interleaved=interleaved, shared=shared)
        return (a * b).sum()

    assert abs(product(pq, pk) - product(pq + shift, pk + shift)) < 1e-10
    assert abs(product(pq, pk) - product(pq + shift, pk)) > 1e-6


def test_interleaved_pairs_are_complex_products_and_the_rest_passes():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 2, 16))
    pos = rng.integers(0, 9, (3, 2))
    y, scale = H.rope_ref(x, pos, [4, 4], theta=100.0)
    for t in range(3):
        f = [1.0, 100.0 ** -0.5]
        phase = np.exp(1j * np.array([pos[t, 0] * f[0], pos[t, 0] * f[1], pos[t, 1] * f[0], pos[t, 1] * f[1]]))
        z = (x[:, t, :, 0:8:2] + 1j * x[:, t, :, 1:8:2]) * phase
        assert np.allclose(y[:, t, :, 0:8:2], z.real) and np.allclose(y[:, t, :, 1:8:2], z.imag)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.all(np.abs(y) <= scale + 1e-12)


def test_shared_ladder_runs_on_over_the_axes():
    a = H.rope_angles(np.array([[2.0, 3.0]]), [4, 4], theta=16.0, shared=True)
    assert np.allclose(a, [[2.0, 2.0 * 16 ** -0.25, 3.0 * 16 ** -0.5, 3.0 * 16 ** -0.75]])


def test_norm_makes_unit_mean_squares():
    x = np.random.default_rng(2).standard_normal((1, 4, 2, 8)) * 7
    y, _ = H.rope_ref(x, np.zeros((4, 1)), [8], weight=np.full(8, 3.0), eps=0.0)
    assert np.allclose((y * y).mean(-1), 9.0)


def test_attention_against_a_loop():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((2, 3, 4, 8)), rng.standard_normal((2, 5, 2, 8)), rng.standard_normal((2, 5, 2, 8))
    o, w = H.attention_ref(q, k, v, kv_lens=[4, 0], scale=0.3)
    assert np.array_equal(o[1], np.zeros((3, 4, 8)))
    for t in range(3):
        for h in range(4):
            e = [np.exp(0.3 * q[0, t, h] @ k[0, j, h // 2]) for j in range(4)]
            want = sum(e[j] * v[0, j, h // 2] for j in range(4)) / sum(e)
            assert np.allclose(o[0, t, h], want)
    assert np.all(np.abs(o) <= w + 1e-12)
