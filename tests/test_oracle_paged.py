"""The paged cache's oracle against closed forms."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import paged as P


@pytest.mark.parametrize("half", [False, True])
def test_rotation(half):
    rng = np.random.default_rng(0)
    x, f = rng.normal(size=(5, 2, 32)), P.frequencies(16, 1e4)
    pos = np.array([0, 1, 7, 100, 5000])
    y, _ = P.norm_rotate(x, None, 0.0, pos, f, half)
    assert np.allclose(y[0], x[0]) and np.array_equal(y[..., 16:], x[..., 16:])
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    # products of two rows go by the distance of their positions
    a, b = (P.norm_rotate(np.stack([x[1], x[2]]), None, 0.0, np.array(p), f, half)[0] for p in ((3, 10), (103, 110)))
    assert np.allclose((a[0] * a[1]).sum(-1), (b[0] * b[1]).sum(-1))
    # the pair of the first frequency turns by one radian a position
    one = np.zeros((1, 1, 32))
    one[0, 0, 0] = 1.0
    z, _ = P.norm_rotate(one, None, 0.0, np.array([1]), f, half)
    assert math.isclose(z[0, 0, 0], math.cos(1.0)) and math.isclose(z[0, 0, 8 if half else 1], math.sin(1.0))


def test_norm():
    x = np.full((1, 1, 64), -3.0)
    y, _ = P.norm_rotate(x, np.arange(64.0), 0.0, np.zeros(1), np.zeros(0), False)
    assert np.allclose(y[0, 0], -np.arange(64.0))


def test_scaled_frequencies():
    f = P.frequencies(64, 1e4)
    assert np.allclose(P.frequencies(64, 1e4, "linear", 4.0), f / 4)
    g = P.frequencies(64, 1e4, "parts", 8.0, 8192)
    turns = 8192 * f / (2 * math.pi)
    assert np.allclose(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((g[mid] < f[mid]) & (g[mid] > f[mid] / 8)).all()


def test_seen():
    assert P.seen(3, 6).tolist() == [1, 1, 1, 1, 0, 0]
    assert P.seen(3, 6, causal=False).all()
    assert P.seen(4, 6, window=2).tolist() == [0, 0, 0, 1, 1, 0]
    assert P.seen(4, 6, window=1, sinks=2).tolist() == [1, 1, 0, 0, 1, 0]
    assert not P.seen(-1, 6).any()


def test_attend():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 2, 8))
    out, mass, _ = P.attend(q, k, v, 0.5)
    for t in range(3):
        for h in range(4):
            w = [math.exp(0.5 * sum(q[t, h, d] * k[j, h // 2, d] for d in range(8))) for j in range(t + 3)]
            for d in range(8):
                assert math.isclose(out[t, h, d], sum(x * v[j, h // 2, d] for j, x in enumerate(w)) / sum(w), abs_tol=1e-12)
    assert (mass >= np.abs(out) - 1e-12).all()
    one, _, _ = P.attend(q[:1], k, v, 0.5, window=1)
    assert np.allclose(one[0], np.repeat(v[4], 2, 0))
    none, _, _ = P.attend(np.ones((3, 4, 8)), k[:2], v[:2], 1.0)
    assert (none[0] == 0).all() and np.allclose(none[1], np.repeat(v[0], 2, 0))
