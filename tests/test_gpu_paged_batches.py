"""Batches of the paged cache whose numbers are wrong or unusual: what a call leaves out, and what it does all the same."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_speculative_decoding_fm_gb300 as fm
from oracle import paged as P
from paged_common import TYPES, Batch, check_attend, half_step
from test_gpu_paged import BLOCKS, CHUNKS, TOKENS

pytestmark = pytest.mark.gpu
INVALID = fm.FM_ERR_INVALID_ARG


def refused(status, call):
    with pytest.raises(fm.FmError) as e:
        call()
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("seqs", [1, 7, 32, 33, 200])
@pytest.mark.parametrize("value", [-1, -2 ** 31, 2 ** 31 - 1, None])
def test_a_bad_start_costs_its_own_sequences(seqs, value):
    """One start outside the packed rows: the write leaves out the sequences that it begins and ends, as the attention does, writes
    the others' rows and reports it.  (None: a length past the table.)"""
    rng = np.random.default_rng(seqs)
    B = Batch([(int(rng.integers(1, 4)), int(rng.integers(0, 30))) for _ in range(seqs)], 1, 2, 64, 16, TYPES["f16"], seed=56, fill=3.0, pad=3)
    B.create(rot_dims=16)
    x = torch.from_numpy(rng.normal(size=(B.total, 4, 64))).half().cuda()
    w = torch.ones(64, device="cuda")

    def write():
        q = torch.full((B.total, 2, 64), 9.0, dtype=B.t, device="cuda")
        B.k_pool.fill_(3.0), B.v_pool.fill_(3.0)
        fm.fm_paged_write(B.c, 0, B.b, x[:, :2], x[:, 2:3], x[:, 3:], q, w, w)
        return q, B.k_pool.clone(), B.v_pool.clone()

    good = write()
    fm.fm_paged_synchronize(B.c)
    first = np.concatenate([[0], np.cumsum(B.n)])
    for i in sorted({0, seqs // 3, seqs // 2, seqs - 1, seqs}):
        saved = B.starts.clone(), B.len_dev.clone()
        if value is None:
            i = min(i, seqs - 1)
            B.len_dev[i] = 2 ** 30
            lost = [i]
        else:
            B.starts[i] = value
            lost = [j for j in (i - 1, i) if 0 <= j < seqs]
        got = write()
        refused(INVALID, lambda: fm.fm_paged_synchronize(B.c))
        want = [y.clone() for y in good]
        for j in lost:
            want[0][first[j]:first[j + 1]] = 9.0
            for p in range(B.lengths[j] - B.n[j], B.lengths[j]):
                for pool in want[1:]:
                    pool[0, int(B.table_np[j, p // 16]), :, p % 16] = 3.0
        for a, b in zip(got, want):
            assert torch.equal(a, b), (i, lost)
        out = torch.full((B.total, 2, 64), 9.0, dtype=B.t, device="cuda")
        fm.fm_paged_attend(B.c, 0, B.b, good[0], out)
        refused(INVALID, lambda: fm.fm_paged_synchronize(B.c))
        left = [t for j in lost for t in range(first[j], first[j + 1])] + list(range(B.total - 3, B.total))
        assert (out == 9.0).flatten(1).all(1).nonzero()[:, 0].tolist() == sorted(left)
        B.starts.copy_(saved[0]), B.len_dev.copy_(saved[1])


def test_both_errors_are_reported():
    """A batch that pointed outside and a wait that gave up: one check reports the wait, the next the batch, then neither; on
    any stream."""
    B = Batch([(2, 30), (1, 5)], 1, 2, 64, 16, TYPES["f16"], seed=57).create().fill_rows()
    q = B.queries()
    out = torch.empty_like(q)
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        B.len_dev[0] = -1
        fm.fm_paged_write(B.c, 0, B.b, q, None, None, out)
        torch.cuda.synchronize()
        fm.fm_paged_selftest_wait_timeout(B.c, 1000, stream=stream)
        refused(fm.FM_ERR_TIMEOUT, lambda: fm.fm_paged_synchronize(B.c, stream=stream))
        refused(INVALID, lambda: fm.fm_paged_synchronize(B.c, stream=stream))
        fm.fm_paged_synchronize(B.c, stream=stream)
        B.len_dev[0] = B.lengths[0]
    fm.fm_paged_write(B.c, 0, B.b, q, None, None, out)
    fm.fm_paged_synchronize(B.c)


def test_threads_report_an_error_once():
    """Four host threads check their streams at the same time: one of them reports."""
    import threading
    B = Batch([(2, 30)], 1, 2, 64, 16, TYPES["f16"], seed=58).create().fill_rows()
    q, streams = B.queries(), [torch.cuda.Stream() for _ in range(4)]
    out = torch.empty_like(q)
    for _ in range(20):
        B.len_dev[0] = -1
        fm.fm_paged_write(B.c, 0, B.b, q, None, None, out)
        torch.cuda.synchronize()
        found, gate = [], threading.Barrier(4)

        def check(s):
            gate.wait()
            try:
                fm.fm_paged_synchronize(B.c, stream=s)
            except fm.FmError as e:
                found.append(e.status)

        threads = [threading.Thread(target=check, args=(s,)) for s in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert found == [INVALID]


KINDS = [(TOKENS, (2, 2, 64)), (BLOCKS, (2, 1, 128)), (CHUNKS, (2, 1, 128)), (CHUNKS, (1, 3, 64)), (CHUNKS, (1, 3, 256)), (BLOCKS, (1, 8, 128))]


@pytest.mark.parametrize("scale", [0.03, 0.5, 1.0])
@pytest.mark.parametrize("seqs,heads", KINDS)
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_scale(seqs, heads, t, scale):
    B = Batch(seqs, *heads, 32, TYPES[t], seed=60).create().fill_rows()
    q = B.queries(0.5)
    out = torch.full_like(q, 7.0)
    fm.fm_paged_attend(B.c, 0, B.b, q, out, scale=scale)
    fm.fm_paged_synchronize(B.c)
    check_attend(B, q, out, scale=scale)


@pytest.mark.parametrize("scale", [1e-30, 1e30])
@pytest.mark.parametrize("seqs,heads", KINDS)
def test_ends_of_the_scale(seqs, heads, scale):
    """All scores equal to rounding: the mean of the rows.  One score far above the others: its row, or the mean of those that share
    it (from 512 on bf16 keys go in steps of 4)."""
    B = Batch(seqs, *heads, 32, TYPES["bf16"], seed=61).create().fill_rows()
    q = torch.ones((B.total, B.heads, B.hd), dtype=B.t, device="cuda")
    B.k_pool.fill_(0.0)
    for i, n in enumerate(B.lengths):       # a row's size is its place: the last seen one is the largest
        for j in range(n):
            B.k_pool[0, int(B.table_np[i, j // 32]), :, j % 32, :2] = float(j + 1) if j < 256 else 256.0 + 2 * (j - 255)
    out = torch.full_like(q, 7.0)
    fm.fm_paged_attend(B.c, 0, B.b, q, out, scale=scale)
    fm.fm_paged_synchronize(B.c)
    got, first = out.double().cpu().numpy(), 0
    for i, n in enumerate(B.n):
        if n:
            ones = np.ones((n, B.heads, B.hd))
            want, mass, _ = P.attend(ones, B.rows(i, B.k_pool), B.rows(i, B.v_pool), scale)
            # (weights are 1, or 0: their sum is exact, the products' sums are off by 2^-20 of the mass, the output by half a step)
            assert (np.abs(got[first:first + n] - want) <= half_step(B.t) * np.abs(want) + 2.0 ** -18 * mass).all()
        first += n


@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 11, 2.0 ** 13, 2.0 ** 15, 2.0 ** 40])
@pytest.mark.parametrize("seqs,heads", KINDS)
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_far_scores(seqs, heads, t, size):
    """Scaled scores from 2^16 on to beyond what an exponent holds, of either sign, in whole numbers that a factor of two separates:
    the largest one's row alone."""
    if t == "f16" and size > 2.0 ** 15:
        pytest.skip("not an f16")
    B = Batch(seqs, *heads, 32, TYPES[t], seed=64).create().fill_rows()
    q = torch.zeros((B.total, B.heads, B.hd), dtype=B.t, device="cuda")
    q[:, :, 0] = size
    for sign in (1.0, -1.0):
        B.k_pool.fill_(0.0)
        for i, n in enumerate(B.lengths):
            steps = torch.randperm(n, generator=torch.Generator().manual_seed(i)).double() % 127 + 129   # (eight bits)
            steps[torch.arange(n) % 9 == 0] = 0.0
            for j in range(n):
                B.k_pool[0, int(B.table_np[i, j // 32]), :, j % 32, 0] = sign * float(steps[j]) * size / 256
        out = torch.full_like(q, 7.0)
        fm.fm_paged_attend(B.c, 0, B.b, q, out, scale=1.0)
        fm.fm_paged_synchronize(B.c)
        got, first = out.double().cpu().numpy(), 0
        for i, n in enumerate(B.n):
            if n:
                want, mass, _ = P.attend(q[first:first + n].double().cpu().numpy(), B.rows(i, B.k_pool), B.rows(i, B.v_pool), 1.0)
                # A weight is not 1 but 2^r, r what rounding reference * scale leaves (up to 2^-24 of it, the same for all weights of a
                # row): its own rounding to the pool's type, half a step, moves the output and not the sum of weights.
                e = half_step(B.t)
                assert (np.abs(got[first:first + n] - want) <= e * np.abs(want) + (e * (1 + e) + 2.0 ** -18) * mass).all(), sign
            first += n


@pytest.mark.parametrize("max_new", [0, 1, 20, 129])
@pytest.mark.parametrize("seqs,heads", [(CHUNKS, (2, 1, 64)), (CHUNKS, (1, 2, 128)), (CHUNKS, (1, 3, 256)), (BLOCKS, (1, 6, 256))])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 5)])
def test_more_rows_than_max_new(seqs, heads, max_new, window, sinks):
    """A sequence with more new rows than the batch says: the kernel that was chosen for fewer attends over all of them."""
    B = Batch(seqs, *heads, 32, TYPES["bf16"], seed=62).create().fill_rows()
    q = B.queries()
    b = fm.fm_paged_batch(B.c, B.starts, B.len_dev, B.table, B.total, max_new)
    out = torch.full_like(q, 7.0)
    fm.fm_paged_attend(B.c, 0, b, q, out, window=window, sinks=sinks)
    fm.fm_paged_synchronize(B.c)
    check_attend(B, q, out, window=window, sinks=sinks)


@pytest.mark.parametrize("heads,new,past", [((1, 1, 128), 40, 4000), ((1, 4, 64), 16, 9000), ((1, 6, 256), 24, 3000)])
def test_long_rows_in_small_tiles(heads, new, past):
    """Tiles of 16 rows over a long sequence, each cut between CTAs."""
    B = Batch([(new, past)], *heads, 64, TYPES["f16"], seed=63).create().fill_rows()
    q = B.queries()
    b = fm.fm_paged_batch(B.c, B.starts, B.len_dev, B.table, B.total, 1)
    for causal in (True, False):
        out = torch.full_like(q, 7.0)
        fm.fm_paged_attend(B.c, 0, b, q, out, causal=causal)
        fm.fm_paged_synchronize(B.c)
        check_attend(B, q, out, causal=causal)
