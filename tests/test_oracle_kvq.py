"""Pins of the 4-bit cache's oracle against hand-made groups, brute force and closed forms."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import kvq as Q


def test_group_by_hand():
    x = np.zeros(32)
    x[:4] = [-8.0, 7.0, 0.5, 1.5]          # d = 1: 0.5 and 1.5 lie on borders, ties to even
    c, d = Q.quantize(x)
    assert d[0] == 1.0 and list(c[:5]) == [0, 15, 8, 10, 8]
    assert list(Q.values(c, d)[:5]) == [-8.0, 7.0, 0.0, 2.0, 0.0]
    c, d = Q.quantize(-x)                  # the scale takes the sign of the largest value
    assert d[0] == -1.0 and list(Q.values(c, d)[:2]) == [8.0, -7.0]
    x[:2] = [8.0, -8.0]                    # a tie goes to the negative value; the positive one saturates at 7 d
    c, d = Q.quantize(x)
    assert d[0] == 1.0 and list(Q.values(c, d)[:2]) == [7.0, -8.0]


def test_extremes():
    x = np.zeros((4, 32))
    x[1, 3], x[1, 4] = np.nan, 2.0
    x[2, 0], x[2, 1] = np.inf, -np.inf
    x[3, 0] = 1e-8                          # the scale rounds to zero
    c, d = Q.quantize(x)
    v = Q.values(c, d)
    assert np.all(v[0] == 0) and v[1, 3] == 0 and v[1, 4] == 2.0
    assert v[2, 1] == -8 * 65504.0 and v[2, 0] == 7 * 65504.0
    assert np.all(v[3] == 0) and np.all(np.isfinite(v))


def test_error_is_half_a_step():
    x = np.random.default_rng(3).normal(size=(50, 64))
    c, d = Q.quantize(x)
    err = np.abs(Q.values(c, d) - x).reshape(50, 2, 32)
    step = np.abs(d.astype(np.float64))[..., None]
    # half a step; up to a whole one where +|m| of the other sign saturates at 7 d; the scale's own rounding moves the
    # largest value by 8 d 2^-11
    assert np.all(err <= step * (1.0 + 8 * 2.0 ** -11))
    inside = np.abs(x).reshape(50, 2, 32) <= 7.5 * step * (1 - 2.0 ** -10)
    assert np.all(err[inside] <= 0.5 * np.broadcast_to(step, err.shape)[inside] + 1e-12)


@pytest.mark.parametrize("causal", [False, True])
def test_attend_brute_force(causal):
    rng = np.random.default_rng(5)
    T, H, hkv, hd, L, first = 3, 4, 2, 8, 6, 1
    q, k, v = rng.normal(size=(T, H, hd)), rng.normal(size=(L, hkv, hd)), rng.normal(size=(L, hkv, hd))
    out, w, mass, reach = Q.attend(q, k, v, 0.3, causal, first)
    want_w = np.zeros((hkv, L))
    for t in range(T):
        for h in range(H):
            js = [j for j in range(first, L) if not causal or j <= L - T + t]
            s = [math.exp(0.3 * sum(q[t, h, d] * k[j, h // 2, d] for d in range(hd))) for j in js]
            for d in range(hd):
                assert abs(out[t, h, d] - sum(a * v[j, h // 2, d] for a, j in zip(s, js)) / sum(s)) < 1e-12
            for a, j in zip(s, js):
                want_w[h // 2, j] += a / sum(s)
    assert np.allclose(w, want_w, atol=1e-12) and abs(w.sum() - T * H) < 1e-9


def test_rows_that_see_nothing():
    q, k = np.ones((4, 1, 8)), np.ones((2, 1, 8))
    out, w, _, _ = Q.attend(q, k, k, 1.0, causal=True)
    assert np.all(out[:2] == 0) and np.all(out[2:] == 1) and np.allclose(w, [[1.5, 0.5]])
    out, w, _, _ = Q.attend(q, k, k, 1.0, first=2)
    assert np.all(out == 0) and np.all(w == 0)


def test_kept_rows():
    w = np.array([1.0, 3.0, 3.0, 0.0, 2.0, 9.0])
    assert list(Q.kept_rows(w, 6, 0)) == [0, 1, 2, 3, 4, 5]
    assert list(Q.kept_rows(w, 3, 1)) == [1, 2, 5]
    assert list(Q.kept_rows(w, 2, 1)) == [1, 5]          # a tie: the lowest row
    assert list(Q.kept_rows(w, 2, 2)) == [4, 5] and list(Q.kept_rows(w, 0, 0)) == []
    assert list(Q.kept_rows(np.array([np.nan, -1.0, -2.0, 0.0]), 3, 0)) == [1, 2, 3]
