"""Pins of the norm's oracle: its gradient against differences, its angles
against a second reduction, and known values."""

import math

import numpy as np
import pytest

from oracle import qk_norm as N


def test_angles_drop_whole_turns_exactly():
    assert abs(N.PI / (1 << N.BITS) - math.pi) < 1e-15
    f = np.array([1.0, 0.5, 1e-5, 0.0, -0.25])
    a = N.angles([0, 1, 3, -2], f)
    want = np.array([0, 1, 3, -2])[:, None] * f
    np.testing.assert_allclose(np.exp(1j * a), np.exp(1j * want), atol=1e-15)
    # 2^31 - 1 radians, by sums of angles: sin and cos of 2^k from those of 2^(k-1)
    z, total = complex(math.cos(1), math.sin(1)), complex(1, 0)
    for _ in range(31):
        total *= z
        z *= z
    np.testing.assert_allclose(np.exp(1j * N.angles([2 ** 31 - 1], [1.0])[0, 0]), total, atol=1e-5)


def test_positions():
    p, there = N.positions(7, [1, 3, 3, 6], [10, 5, 2])
    assert p.tolist() == [0, 8, 9, -1, 0, 1, 0] and there.tolist() == [False] + [True] * 5 + [False]
    assert N.positions(3, None, 9)[0].tolist() == [6, 7, 8]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_gradient_against_differences(interleaved, weighted):
    rng = np.random.default_rng(0)
    T, H, d, rot = 3, 2, 32, 16
    x, dz = rng.normal(size=(2, T, H, d))
    w = rng.normal(size=d) if weighted else None
    f, pos, eps = 0.5 ** np.arange(rot // 2), [0, 7, -3], 1e-2
    dx, dw, _, _ = N.backward(x, dz, pos, w, eps, f, interleaved)

    def loss(x, w):
        return (N.forward(x, pos, w, eps, f, interleaved)[0] * dz).sum()

    h = 1e-6
    for at in [(0, 0, 0), (1, 1, 5), (2, 0, 31), (1, 0, 16), (2, 1, 15)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-8
        if weighted:
            e = np.zeros(d)
            e[at[2]] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[at[2]]) < 1e-8


def test_a_head_of_one_value_has_norm_one():
    z, _ = N.forward(np.full((1, 1, 64), -3.0), [0], np.ones(64), 1e-12, [1.0] * 8, False)
    np.testing.assert_allclose(z, -1.0)
