"""Pins of the rotary-position oracle: closed forms and invariants."""
import math

import numpy as np
import pytest

from oracle import rope as orope

RNG = np.random.default_rng(5)


@pytest.mark.parametrize("layout", [orope.HALF, orope.INTERLEAVED])
def test_quarter_turn_and_tail(layout):
    x = RNG.standard_normal((1, 2, 8))
    w = np.array([math.pi / 2, math.pi])  # rot 4 of 8
    y = orope.apply(x, np.array([1]), w, layout)
    a, b = orope.pair_index(4, layout)
    np.testing.assert_allclose(y[..., a[0]], -x[..., b[0]], atol=1e-15)  # a quarter turn
    np.testing.assert_allclose(y[..., b[0]], x[..., a[0]], atol=1e-15)
    np.testing.assert_allclose(y[..., a[1]], -x[..., a[1]], atol=1e-15)  # a half turn
    np.testing.assert_allclose(y[..., b[1]], -x[..., b[1]], atol=1e-15)
    assert np.array_equal(y[..., 4:], x[..., 4:])


@pytest.mark.parametrize("layout", [orope.HALF, orope.INTERLEAVED])
def test_relative_positions_norms_and_transpose(layout):
    w = orope.frequencies(10000.0, 32)
    q, k = RNG.standard_normal((1, 1, 64)), RNG.standard_normal((1, 1, 64))
    at = lambda x, p: orope.apply(x, np.array([p]), w, layout)  # noqa: E731
    dots = [float(np.sum(at(q, p + 7) * at(k, p))) for p in (0, 5, 1000, -40)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)  # only the distance matters
    y = orope.apply(q, np.array([77]), w, layout, scale=1.3)
    np.testing.assert_allclose(np.linalg.norm(y[..., :32]), 1.3 * np.linalg.norm(q[..., :32]))
    back = orope.apply(at(q, 77), np.array([77]), w, layout, transpose=True)
    np.testing.assert_allclose(back, q, atol=1e-12)
    # <R x, g> = <x, R^T g>: the transpose is the gradient
    g = RNG.standard_normal(q.shape)
    fwd = orope.apply(q, np.array([9]), w, layout, scale=0.7)
    bwd = orope.apply(g, np.array([9]), w, layout, scale=0.7, transpose=True)
    np.testing.assert_allclose(np.sum((fwd - np.concatenate([0 * q[..., :32], q[..., 32:]], -1)) * g)
                               + np.sum(q[..., 32:] * g[..., 32:]), np.sum(q * bwd), rtol=1e-10)


def test_scalings():
    w = orope.frequencies(10000.0, 64)
    assert w[0] == 1.0 and abs(w[-1] - 10000.0 ** (-62 / 64)) < 1e-12
    np.testing.assert_allclose(orope.frequencies(10000.0, 64, "linear", 4.0), w / 4)
    b = orope.frequencies(10000.0, 64, "base", 8.0)
    assert b[0] == 1.0
    np.testing.assert_allclose(b[-1], w[-1] / 8)  # the slowest pair is slowed by the factor
    p = orope.frequencies(10000.0, 64, "by_parts", 8.0, 4096, 1.0, 32.0)
    turns = 4096 * w / (2 * math.pi)
    np.testing.assert_allclose(p[turns >= 32], w[turns >= 32])
    np.testing.assert_allclose(p[turns <= 1], w[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all((p[mid] < w[mid]) & (p[mid] > w[mid] / 8))
    assert orope.frequencies(500.0, 2, "base", 8.0).tolist() == [1.0]
