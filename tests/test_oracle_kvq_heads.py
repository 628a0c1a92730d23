"""The oracle's attention by matrix products against its plain loops (both 64 bits: they differ by summation order)."""
import numpy as np
import pytest

from oracle import kvq as Q


@pytest.mark.parametrize("T,L,first,causal", [(1, 1, 0, False), (3, 70, 0, True), (9, 5, 0, True), (4, 33, 20, True),
                                              (2, 40, 40, False), (5, 64, 63, False), (0, 9, 0, True), (3, 0, 0, False)])
@pytest.mark.parametrize("hkv,group,hd", [(2, 3, 64), (1, 1, 128)])
def test_same_as_loops(T, L, first, causal, hkv, group, hd):
    rng = np.random.default_rng(T * 100 + L)
    q = rng.normal(size=(T, hkv * group, hd))
    k, v = (Q.stored(rng.normal(size=(L, hkv, hd))) for _ in range(2))
    for scale in (0.125, -0.5):
        a = Q.attend(q, k, v, scale, causal, first)
        b = Q.attend_heads(q, k, v, scale, causal, first)
        for x, y in zip(a, b):
            # sums of at most 128 + 70 terms near 1: 200 x 2^-53 of scores up to ~30, and of the values
            assert x.shape == y.shape and np.allclose(x, y, rtol=1e-11, atol=1e-12)
