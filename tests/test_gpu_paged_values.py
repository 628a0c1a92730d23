"""Infinities and NaN that the paged cache's attention meets, in units of work that one CTA does and in those that are cut between
CTAs and joined."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_speculative_decoding_fm_gb300 as fm
from oracle import paged as P
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


# (seqs, new, past), heads, page, window, sinks
SERVING = [((32, 1, 2000), (4, 6, 256), 64, 0, 0), ((32, 9, 2000), (16, 1, 128), 16, 0, 0), ((8, 700, 300), (4, 6, 256), 64, 0, 0),
           ((8, 700, 2000), (8, 4, 64), 64, 500, 16), ((32, 1, 3000), (8, 4, 64), 64, 500, 4)]


@pytest.mark.parametrize("seqs,heads,page,window,sinks", SERVING)
def test_time_of_garbage_in_hidden_rows(seqs, heads, page, window, sinks):
    """What the rows behind a sequence's end hold costs little time, as it has no part in the result: their infinities and NaN are
    taken out of a tile in one more pass over it.  (Asked for at the unit's end, as those of seen rows are, they took up to 220
    times a call's time.)"""
    n, new, past = seqs
    B = Batch([(new, past + i) for i in range(n)], *heads, page, TYPES["bf16"], seed=54, fill=0.0).create().fill_rows()
    q = B.queries()
    us, outs = [], []
    for x in (0.0, float("nan")):
        for pool in (B.k_pool, B.v_pool):
            for i, m in enumerate(B.lengths):
                if m % page:
                    pool[0, int(B.table_np[i, m // page]), :, m % page:] = x
        outs.append(attend(B, q, window=window, sinks=sinks))
        out, times = torch.empty_like(q), []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(2000000)      # (the calls are queued before they run)
            a.record()
            for _ in range(4):
                fm.fm_paged_attend(B.c, 0, B.b, q, out, window=window, sinks=sinks)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        us.append(sorted(times)[4] * 250)
    assert torch.equal(*outs)
    assert us[1] < 2 * us[0], us


@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads,new", [((2, 2, 64), 3), ((1, 6, 256), 2), ((1, 2, 128), 40), ((1, 2, 64), 200), ((1, 3, 256), 90)])
def test_infinite_values(heads, new, t, page, window, sinks):
    """Infinities and NaN of V, one to a few a column, in rows all over a sequence: each output is infinite or NaN just where
    the sum over the rows that it sees is (small queries: no weight underflows)."""
    B = Batch([(new, 400), (new, 90)], *heads, page, TYPES[t], seed=55).create().fill_rows()
    q = B.queries(0.1)
    for i, n in enumerate(B.lengths):
        for j in list(range(n - new, n)) + [int(x) for x in B.rng.integers(0, n, size=12)]:
            for x in (float("inf"), float("-inf"), float("nan")):
                d = B.rng.integers(0, B.hd, size=1 + B.hd // 64)
                B.v_pool[0, int(B.table_np[i, j // page]), int(B.rng.integers(0, B.kv)), j % page, torch.from_numpy(d).cuda()] = x
    got = attend(B, q, window=window, sinks=sinks).double().cpu().numpy()
    qn, first = q.double().cpu().numpy(), 0
    for i, n in enumerate(B.n):
        with np.errstate(invalid="ignore"):
            want, _, _ = P.attend(qn[first:first + n], B.rows(i, B.k_pool), B.rows(i, B.v_pool), B.hd ** -0.5, True, window, sinks)
        for test in (np.isnan, np.isposinf, np.isneginf):
            assert np.array_equal(test(got[first:first + n]), test(want)), test.__name__
        assert np.isfinite(want).any() and np.isinf(want).any() and np.isnan(want).any()
        first += n
