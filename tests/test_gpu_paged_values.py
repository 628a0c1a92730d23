"""Infinities and NaN that the paged cache's attention meets, in units of work that one CTA does and in those that are cut between
CTAs and joined."""
from __future__ import annotations

import pytest
import torch

from paged_common import TYPES, Batch
from test_gpu_paged import attend

pytestmark = pytest.mark.gpu

# heads, new rows and the rows before them: each kernel (few rows; one tile; two tiles), cut and whole
CUT = [((2, 1, 64), 1, 30000), ((1, 1, 128), 16, 20000), ((1, 8, 256), 2, 20001), ((1, 1, 64), 140, 9000), ((1, 1, 128), 100, 9000),
       ((1, 2, 128), 70, 9100), ((1, 2, 256), 60, 8000)]
WHOLE = [(heads, new, 30) for heads, new, _ in CUT]


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads,new,past", CUT + WHOLE)
def test_nan_query(heads, new, past, t):
    """A query that holds a NaN gives a row of NaN, and changes no bit of the others."""
    B = Batch([(new, past), (new, past)], *heads, 128, TYPES[t], seed=51).create().fill_rows()
    q = B.queries()
    want = attend(B, q)
    for token, head in ((0, 0), (new - 1, B.heads - 1), (2 * new - 1, 0)):
        x = q.clone()
        x[token, head, 3] = float("nan")
        got = attend(B, x)
        assert got[token, head].isnan().all()
        got[token, head] = want[token, head]
        assert torch.equal(got, want)


@pytest.mark.parametrize("heads,new,past", CUT + WHOLE)
def test_nan_keys(heads, new, past):
    """Where every key is NaN, so is every output of the KV head; the other sequence's stay as they are."""
    B = Batch([(new, past), (new, past)], *heads, 128, TYPES["bf16"], seed=52).create().fill_rows()
    q = B.queries()
    want = attend(B, q)
    for j in range(0, new + past, 128):
        B.k_pool[0, int(B.table_np[0, j // 128]), 0] = float("nan")
    got = attend(B, q)
    assert got[:new, :heads[1]].isnan().all()
    assert torch.equal(got[new:], want[new:]) and torch.equal(got[:, heads[1]:], want[:, heads[1]:])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads,new,past", CUT + WHOLE)
def test_scores_of_minus_infinity(heads, new, past, t):
    """Keys whose scores are minus infinity have no weight, as those far below the others have none; a row that sees nothing
    else is 0 / 0, and one that sees nothing stays zeros."""
    B = Batch([(new, past), (new, -new)], *heads, 128, TYPES[t], seed=53).create().fill_rows()
    q = B.queries().abs() + 0.5
    few = past // 2
    outs = []
    for x in (float("-inf"), -30000.0):
        for j in range(0, few, 128):
            B.k_pool[0, int(B.table_np[0, j // 128]), :, :few - j] = x
        outs.append(attend(B, q))
    assert torch.equal(outs[0], outs[1]) and outs[0].isfinite().all() and (outs[0][new:] == 0).all()
    for j in range(0, new + past, 128):
        B.k_pool[0, int(B.table_np[0, j // 128])] = float("-inf")
    got = attend(B, q)
    assert got[:new].isnan().all() and (got[new:] == 0).all()
