"""Calls on the paged cache beside the plain ones: refusals, what is masked, stale and bad pages, graphs that are replayed with
other lengths and pages, streams, strides, far pools, and a write followed by the attention that reads it."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import block_speculative_decoding_fm_gb300 as fm
from oracle import paged as P
from paged_common import TYPES, Batch, check_attend, half_step
from test_gpu_paged import BLOCKS, CHUNKS, TOKENS, attend

pytestmark = pytest.mark.gpu
INVALID, UNSUPPORTED = fm.FM_ERR_INVALID_ARG, fm.FM_ERR_UNSUPPORTED


def refused(status, call):
    with pytest.raises(fm.FmError) as e:
        call()
    assert e.value.status == status, str(e.value)


SHAPES = [(TOKENS, (2, 2, 64), 16), (BLOCKS, (2, 1, 128), 64), (CHUNKS, (2, 1, 128), 32), (CHUNKS, (1, 3, 256), 128), (CHUNKS, (1, 5, 64), 16)]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_masked_rows_hold_anything(shape, t):
    """Infinities and NaN in rows that a row does not see change no bit of its output; rows that see them show them."""
    seqs, heads, page = SHAPES[shape]
    B = Batch(seqs, *heads, page, TYPES[t], seed=20, fill=1.0).create().fill_rows()
    q = B.queries()
    for kw in (dict(), dict(window=50, sinks=3)):
        clean = attend(B, q, **kw)
        k0, v0 = B.k_pool.clone(), B.v_pool.clone()
        first = 0
        for i, (n, past) in enumerate(seqs):
            if n < 2 or B.lengths[i] < 2:
                first += n
                continue
            # the last new row: seen by itself alone
            j = B.lengths[i] - 1
            for pool, x in ((B.k_pool, float("nan")), (B.v_pool, float("inf"))):
                pool[0, int(B.table_np[i, j // page]), 0, j % page, ::3] = x
            got = attend(B, q, **kw)
            assert torch.equal(got[:first + n - 1], clean[:first + n - 1]) and torch.equal(got[first + n:], clean[first + n:])
            assert not torch.isfinite(got[first + n - 1, 0].float()).any()
            assert torch.equal(got[first + n - 1, heads[1]:], clean[first + n - 1, heads[1]:])
            B.k_pool.copy_(k0)
            B.v_pool.copy_(v0)
            # V alone: the columns that hold it
            B.v_pool[0, int(B.table_np[i, j // page]), 0, j % page, 5] = float("-inf")
            got = attend(B, q, **kw)
            assert torch.equal(got[:first + n - 1], clean[:first + n - 1])
            row = got[first + n - 1, :heads[1]].float()
            assert (row[:, 5] == float("-inf")).all()
            assert torch.equal(row[:, 6:], clean[first + n - 1, :heads[1], 6:].float())
            B.v_pool.copy_(v0)
            first += n


@pytest.mark.parametrize("heads,new", [((2, 1, 64), 1), ((1, 2, 128), 5), ((1, 2, 128), 150), ((1, 1, 256), 40)])
def test_pages_behind_the_window_may_be_gone(heads, new):
    """Table entries of pages that no row of the call sees may point anywhere."""
    B = Batch([(new, 700), (new, 300)], *heads, 16, TYPES["bf16"], seed=21).create().fill_rows()
    q = B.queries()
    want = attend(B, q, window=100, sinks=20)
    for i, n in enumerate(B.lengths):
        seen = np.zeros(n, bool)
        for p in range(n - new, n):
            seen |= P.seen(p, n, True, 100, 20)
        for page in range(-(-n // 16)):
            if not seen[16 * page:16 * page + 16].any():
                B.table[i, page] = -123456 if page % 2 else 2 ** 30
    assert torch.equal(want, attend(B, q, window=100, sinks=20))


def test_bad_numbers_are_reported():
    """A page outside the pool reads as zeros; starts and lengths outside leave the sequence out; both are reported, once."""
    for heads, new in (((2, 1, 64), 1), ((1, 1, 128), 40)):
        B = Batch([(new, 100), (new, 60)], *heads, 16, TYPES["f16"], seed=22).create().fill_rows()
        q = B.queries()
        good = attend(B, q)
        for edit, left in ((lambda: B.table[0].__setitem__(1, B.pages), False), (lambda: B.table[0].__setitem__(0, -1), False),
                           (lambda: B.len_dev.__setitem__(0, 17 * 1000), True), (lambda: B.len_dev.__setitem__(0, -1), True),
                           (lambda: B.starts.__setitem__(0, -1), True)):
            saved = B.table.clone(), B.len_dev.clone(), B.starts.clone()
            edit()
            out = torch.full_like(q, 7.0)
            fm.fm_paged_attend(B.c, 0, B.b, q, out)
            refused(INVALID, lambda: fm.fm_paged_synchronize(B.c))
            fm.fm_paged_synchronize(B.c)
            assert torch.equal(out[new:], good[new:])
            if left:
                assert (out[:new] == 7.0).all()
            for x, y in zip((B.table, B.len_dev, B.starts), saved):
                x.copy_(y)
        assert torch.equal(good, attend(B, q))


def test_write_reports_bad_pages():
    B = Batch([(3, 30), (2, 5)], 1, 1, 64, 16, TYPES["f16"], seed=23, fill=1.0).create()
    x = torch.randn((5, 1, 64), device="cuda")
    out = torch.full((5, 1, 64), 7.0, dtype=torch.float16, device="cuda")
    B.table[0, 2] = B.pages
    before = B.k_pool.clone()
    fm.fm_paged_write(B.c, 0, B.b, x, x, x, out)
    refused(INVALID, lambda: fm.fm_paged_synchronize(B.c))
    rows = B.rows(1, B.k_pool)[5:]
    assert np.allclose(rows[:, 0], x[3:, 0].half().double().cpu().numpy())
    assert (B.k_pool != before).sum() <= (2 + 2) * 64, "rows of pages that are there"
    assert torch.equal(out, x.half())          # (queries need no page)
    B.len_dev[1] = 1                           # more new rows than rows: the first has no place
    out.fill_(7.0)
    fm.fm_paged_write(B.c, 0, B.b, x, None, None, out)
    refused(INVALID, lambda: fm.fm_paged_synchronize(B.c))
    assert (out[3] == 7.0).all() and torch.equal(out[4], x[4].half())


def test_more_new_rows_than_rows():
    """Rows at negative positions see nothing and give zeros."""
    for heads, n in (((2, 1, 64), 3), ((1, 8, 128), 40)):
        B = Batch([(n, -2), (n, 5), (n, -n)], *heads, 16, TYPES["bf16"], seed=24).create().fill_rows()
        q = B.queries()
        got = attend(B, q)
        check_attend(B, q, got)
        assert (got[:2] == 0).all() and (got[2 * n:] == 0).all()


def test_replay_with_other_lengths_and_pages():
    """A captured call reads starts, lengths and pages when it is replayed; two graphs and eager calls run side by side."""
    heads = (2, 2, 128)
    A = Batch([(3, 200), (1, 90), (5, 7)], *heads, 32, TYPES["bf16"], seed=25, cols=20, pad=4, spare=20).create().fill_rows()
    Z = Batch([(4, 300), (0, 0), (2, 31)], *heads, 32, TYPES["bf16"], seed=26, cols=20, pad=7).create().fill_rows()
    assert Z.pages <= A.pages and Z.total == A.total
    q = A.queries()
    b = fm.fm_paged_batch(A.c, A.starts, A.len_dev, A.table, A.total, 40)
    outs, graphs = [torch.full_like(q, 7.0) for _ in range(2)], []
    fm.fm_paged_attend(A.c, 0, b, q, torch.empty_like(q))
    for out in outs:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            fm.fm_paged_attend(A.c, 0, b, q, out)
        graphs.append(g)
    other = torch.cuda.Stream()
    for g, s in zip(graphs, (torch.cuda.current_stream(), other)):
        with torch.cuda.stream(s):
            for _ in range(5):
                g.replay()
    eager = torch.full_like(q, 7.0)
    fm.fm_paged_attend(A.c, 0, b, q, eager)
    torch.cuda.synchronize()
    rows = sum(A.n)
    for out in outs + [eager]:
        assert torch.equal(out[:rows], eager[:rows]) and (out[rows:] == 7.0).all()
    check_attend(A, q, eager)
    # other sequences in the same places
    A.k_pool[:, :Z.pages], A.v_pool[:, :Z.pages] = Z.k_pool, Z.v_pool
    A.starts.copy_(Z.starts), A.len_dev.copy_(Z.len_dev), A.table.copy_(Z.table)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        check_attend(Z, q, out)
    fm.fm_paged_synchronize(A.c)


def test_write_then_attend_by_chunks():
    """A prompt in chunks of any sizes, then tokens, each written and attended over in turn, as a graph and without: what one
    causal pass over all of it gives."""
    kv, group, hd, page, n = 2, 3, 64, 16, 300
    rng = np.random.default_rng(27)
    rope = dict(rot_dims=32, layout=fm.FM_ROPE_HALF, theta=1e4, scaling=fm.FM_ROPE_LINEAR, factor=2.0)
    x = torch.from_numpy(rng.normal(size=(n, kv * group + 2 * kv, hd))).half().cuda()
    wq, wk = (torch.from_numpy(1 + 0.1 * rng.normal(size=hd)).float().cuda() for _ in "qk")
    table = torch.from_numpy(rng.permutation(20).astype(np.int32)).cuda()[None]
    out = torch.zeros((n, kv * group, hd), dtype=torch.float16, device="cuda")
    k_pool = torch.full((1, 20, kv, page, hd), float("nan"), dtype=torch.float16, device="cuda")
    c = fm.fm_paged_create(k_pool, torch.full_like(k_pool, float("nan")), kv * group, **rope)
    at = 0
    for m in (1, 17, 100, 2, 128, 1, 1, 50):
        part = x[at:at + m]
        starts, lengths = torch.tensor([0, m], dtype=torch.int32, device="cuda"), torch.tensor([at + m], dtype=torch.int32, device="cuda")
        b = fm.fm_paged_batch(c, starts, lengths, table, m)
        q = torch.empty((m, kv * group, hd), dtype=torch.float16, device="cuda")
        fm.fm_paged_write(c, 0, b, part[:, :kv * group], part[:, kv * group:kv * group + kv], part[:, kv * group + kv:], q, wq, wk)
        fm.fm_paged_attend(c, 0, b, q, out[at:at + m])
        at += m
    fm.fm_paged_synchronize(c)
    f = P.frequencies(32, 1e4, "linear", 2.0)
    d = x.double().cpu().numpy()
    q, _ = P.norm_rotate(d[:, :kv * group], wq.cpu().numpy(), 1e-6, np.arange(n), f, True)
    k, _ = P.norm_rotate(d[:, kv * group:kv * group + kv], wk.cpu().numpy(), 1e-6, np.arange(n), f, True)
    v = d[:, kv * group + kv:]
    want, mass, reach = P.attend(q, k, v, hd ** -0.5)
    # q and k are rounded once more here: a score moves by 2^-11 of each of its factors' magnitudes
    e = half_step(torch.float16)
    bound = e * np.abs(want) + (e + 2 * reach[..., None] * (2 * e + 2.0 ** -20) * 1.1) * mass + n * 2.0 ** -25 * np.abs(v).max()
    off = np.abs(out.double().cpu().numpy() - want) / bound
    assert off.max() <= 1.0, off.max()


def test_strides_and_places():
    """Queries out of a projection's rows, outputs into a wider row, queries rotated in place."""
    B = Batch([(20, 100), (1, 30)], 2, 2, 64, 16, TYPES["bf16"], seed=28).create(rot_dims=64).fill_rows()
    q = B.queries()
    want = attend(B, q)
    wide = torch.zeros((B.total, 4 + 3, 2, 64), dtype=B.t, device="cuda")
    wide[:, :4, 1] = q
    out = torch.full((B.total, 9, 64 + 8), 7.0, dtype=B.t, device="cuda")
    fm.fm_paged_attend(B.c, 0, B.b, wide[:, :4, 1], out[:, 2:6, :64])
    fm.fm_paged_synchronize(B.c)
    assert torch.equal(out[:, 2:6, :64], want)
    rest = out.clone()
    rest[:, 2:6, :64] = 7.0
    assert (rest == 7.0).all()
    a, b = torch.empty_like(q), q.clone()
    fm.fm_paged_write(B.c, 0, B.b, q, None, None, a)
    fm.fm_paged_write(B.c, 0, B.b, b, None, None, b)
    fm.fm_paged_synchronize(B.c)
    assert torch.equal(a, b) and not torch.equal(a, q)


def test_other_streams():
    """Calls on a stream that is not the current one, by handle and by object, each with a workspace of its own."""
    B = Batch([(1, 5000)] * 3, 1, 4, 128, 64, TYPES["f16"], seed=29).create().fill_rows()
    q = B.queries()
    want = attend(B, q)
    outs = []
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(12):
        out = torch.full_like(q, 7.0)
        torch.cuda.synchronize()
        s = streams[i % 3]
        fm.fm_paged_attend(B.c, 0, B.b, q, out, stream=s if i % 2 else s.cuda_stream)
        outs.append(out)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


def test_far_pool():
    """Rows past 2^31 elements of the pool."""
    page, kv, hd = 256, 2, 256
    pages = 2 ** 31 // (kv * page * hd) + 40
    k_pool, v_pool = (torch.empty((1, pages, kv, page, hd), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = [pages - 1, 3, pages - 20, pages - 7]
    for i in ids:
        for pool in (k_pool, v_pool):
            pool[0, i] = torch.randn((kv, page, hd), generator=g, device="cuda").bfloat16()
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    small_k, small_v = k_pool[:, ids].contiguous(), v_pool[:, ids].contiguous()
    near = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    for n in (1, 300):
        starts, lengths = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([1000], dtype=torch.int32, device="cuda")
        x = torch.randn((n, 4 + 2 * kv, hd), generator=g, device="cuda").bfloat16()
        res = []
        for k, v, t in ((k_pool, v_pool, table), (small_k, small_v, near)):
            c = fm.fm_paged_create(k, v, 4, rot_dims=64)
            b = fm.fm_paged_batch(c, starts, lengths, t, n)
            q, out = torch.empty((n, 4, hd), dtype=torch.bfloat16, device="cuda"), torch.empty((n, 4, hd), dtype=torch.bfloat16, device="cuda")
            fm.fm_paged_write(c, 0, b, x[:, :4], x[:, 4:6], x[:, 6:], q)
            fm.fm_paged_attend(c, 0, b, q, out)
            fm.fm_paged_synchronize(c)
            res.append((q, out))
        assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
        assert torch.equal(k_pool[:, ids], small_k) and torch.equal(v_pool[:, ids], small_v)


def test_extreme_scores():
    """Scores of every size: one key that outweighs all, equal keys, references that move with every tile."""
    for heads, n in (((1, 1, 64), 1), ((1, 1, 128), 40), ((1, 1, 256), 30)):
        B = Batch([(n, 600)], *heads, 32, TYPES["bf16"], seed=30).create().fill_rows()
        rows = torch.from_numpy(B.rows(0, B.k_pool)).cuda()
        for grow in (torch.linspace(0.0, 40.0, rows.shape[0], dtype=torch.float64), torch.linspace(40.0, 0.0, rows.shape[0], dtype=torch.float64)):
            k = torch.ones_like(rows) * grow.cuda()[:, None, None]
            for j in range(0, rows.shape[0], 32):
                m = min(32, rows.shape[0] - j)
                B.k_pool[0, int(B.table_np[0, j // 32]), :, :m] = k[j:j + m].transpose(0, 1).to(B.t)
            for scale in (-1.0, 0.0, 1.0, 6.0):
                q = torch.full((n, 1, heads[2]), scale, dtype=B.t, device="cuda")
                check_attend(B, q, attend(B, q))


def test_workspace_and_empty_batches():
    B = Batch([(1, 100)], 2, 1, 64, 16, TYPES["f16"], seed=31).create().fill_rows()
    q = B.queries()
    want = attend(B, q)
    need = B.b.workspace_bytes
    assert need == fm.fm_paged_workspace_bytes(B.c, 1) <= fm.fm_paged_workspace_bytes(B.c, 100) <= fm.fm_paged_workspace_bytes(B.c, 1000)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    fm.fm_paged_attend(B.c, 0, B.b, q, out, workspace=ws)
    assert torch.equal(out, want) and (ws[need:] == 255).all()
    refused(INVALID, lambda: fm.fm_paged_attend(B.c, 0, B.b, q, out, workspace=ws[:need - 16]))
    refused(INVALID, lambda: fm.fm_paged_attend(B.c, 0, B.b, q, out, workspace=ws[8:]))
    empty = torch.empty((0,), dtype=torch.int32, device="cuda")
    none = fm.fm_paged_batch(B.c, torch.zeros((1,), dtype=torch.int32, device="cuda"), empty, torch.empty((0, 3), dtype=torch.int32, device="cuda"), 0)
    fm.fm_paged_attend(B.c, 0, none, q[:0], out[:0])
    fm.fm_paged_write(B.c, 0, none, q[:0], None, None, out[:0])
    padded = fm.fm_paged_batch(B.c, torch.zeros((2,), dtype=torch.int32, device="cuda"), torch.zeros((1,), dtype=torch.int32, device="cuda"),
                               torch.zeros((1, 0), dtype=torch.int32, device="cuda"), 1)
    out.fill_(7.0)
    fm.fm_paged_attend(B.c, 0, padded, q, out)
    fm.fm_paged_write(B.c, 0, padded, q, None, None, out)
    fm.fm_paged_synchronize(B.c)
    assert (out == 7.0).all()


def test_refusals():
    B = Batch([(2, 30)], 2, 1, 64, 16, TYPES["f16"], seed=32).create().fill_rows()
    c, b, q = B.c, B.b, B.queries()
    out = torch.empty_like(q)
    k = torch.empty((2, 2, 64), dtype=B.t, device="cuda")
    for call in (lambda: fm.fm_paged_attend(c, 1, b, q, out), lambda: fm.fm_paged_attend(c, -1, b, q, out),
                 lambda: fm.fm_paged_attend(c, 0, b, q, q), lambda: fm.fm_paged_attend(c, 0, b, q, out, scale=0.0),
                 lambda: fm.fm_paged_attend(c, 0, b, q, out, scale=float("nan")), lambda: fm.fm_paged_attend(c, 0, b, q, out, scale=-1.0),
                 lambda: fm.fm_paged_attend(c, 0, b, q, out, scale=1e-38), lambda: fm.fm_paged_attend(c, 0, b, q, out, scale=float("inf")),
                 lambda: fm.fm_paged_attend(c, 0, b, q, out, window=-1), lambda: fm.fm_paged_attend(c, 0, b, q, out, sinks=1),
                 lambda: fm.fm_paged_attend(c, 0, b, q, out, causal=False, window=4), lambda: fm.fm_paged_attend(c, 0, b, q, out, window=4, sinks=-1),
                 lambda: fm.fm_paged_write(c, 0, b), lambda: fm.fm_paged_write(c, 0, b, q), lambda: fm.fm_paged_write(c, 0, b, None, k),
                 lambda: fm.fm_paged_write(c, 0, b, q, k, None, out), lambda: fm.fm_paged_write(c, 3, b, q, None, None, out)):
        refused(INVALID, call)
    wide = torch.empty((2, 2, 70), dtype=B.t, device="cuda")
    refused(INVALID, lambda: fm.fm_paged_attend(c, 0, b, wide[:, :, :64], out))          # rows 140 bytes apart
    refused(INVALID, lambda: fm.fm_paged_attend(c, 0, b, q, torch.empty((2, 2, 72), dtype=B.t, device="cuda")[:, :, 4:68]))
    f32 = torch.empty((2, 2, 64), device="cuda")
    refused(INVALID, lambda: fm.fm_paged_write(c, 0, b, f32, None, None, f32.view(B.t)[:, :, :64]))   # in place, another type
    for call in (lambda: fm.fm_paged_attend(c, 0, b, q.float(), out), lambda: fm.fm_paged_attend(c, 0, b, q[:, :1], out),
                 lambda: fm.fm_paged_attend(c, 0, b, q[:1], out), lambda: fm.fm_paged_attend(c, 0, b, q.cpu(), out),
                 lambda: fm.fm_paged_attend(c, 0, b, q.transpose(1, 2).contiguous().transpose(1, 2), out),
                 lambda: fm.fm_paged_write(c, 0, b, q, k.float(), k, out), lambda: fm.fm_paged_write(c, 0, b, q, None, None, out, f32[0, 0, :32]),
                 lambda: fm.fm_paged_batch(c, B.starts, B.len_dev, B.table.long(), 2), lambda: fm.fm_paged_batch(c, B.starts[:1], B.len_dev, B.table, 2),
                 lambda: fm.fm_paged_batch(c, B.starts, B.len_dev, B.table.cpu(), 2),
                 lambda: fm.fm_paged_create(B.k_pool[0], B.v_pool[0], 2), lambda: fm.fm_paged_create(B.k_pool, B.v_pool.float(), 2),
                 lambda: fm.fm_paged_create(B.k_pool.transpose(2, 3), B.v_pool.transpose(2, 3), 2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        fm.fm_paged_attend(Batch([(2, 3)], 2, 1, 64, 16, B.t).create().c, 0, b, q, out)
    lib = fm.load_library()
    g = fm.FmPagedBatch()
    r = fm.FmPagedRows(q.data_ptr(), 128, 64)
    o = fm.FmPagedRows(out.data_ptr(), 128, 64)

    def raw(**change):
        for f, _ in fm.FmPagedBatch._fields_:
            setattr(g, f, change.get(f, getattr(b.arg, f)))
        ws = torch.empty((b.workspace_bytes,), dtype=torch.uint8, device="cuda")
        return lib.fm_paged_attend(c, 0, ctypes.byref(g), ctypes.byref(r), ctypes.byref(o), 1.0, 1, 0, 0, ws.data_ptr(), ws.numel(), None)

    torch.cuda.synchronize()
    assert raw() == fm.FM_OK
    for change in (dict(n_seqs=-1), dict(n_tokens=-1), dict(max_new=-1), dict(table_pages=-1), dict(starts=None), dict(lengths=None),
                   dict(table=None), dict(table_ld=1, table_pages=2), dict(starts=b.arg.starts + 2)):
        assert raw(**change) == INVALID, change
    for change in (dict(n_seqs=65537), dict(n_tokens=2 ** 31 - 1), dict(table_pages=2 ** 27, table_ld=2 ** 27)):
        assert raw(**change) == UNSUPPORTED, change
    assert lib.fm_paged_attend(c, 0, None, ctypes.byref(r), ctypes.byref(o), 1.0, 1, 0, 0, out.data_ptr(), 1, None) == INVALID
    assert lib.fm_paged_attend(c, 0, ctypes.byref(b.arg), None, ctypes.byref(o), 1.0, 1, 0, 0, out.data_ptr(), 1, None) == INVALID
    torch.cuda.synchronize()


def test_a_wait_that_gives_up_is_reported():
    B = Batch([(1, 10)], 1, 1, 64, 16, TYPES["f16"], seed=33).create().fill_rows()
    fm.fm_paged_selftest_wait_timeout(B.c, 1000)
    refused(fm.FM_ERR_TIMEOUT, lambda: fm.fm_paged_synchronize(B.c))
    fm.fm_paged_synchronize(B.c)
    q = B.queries()
    check_attend(B, q, attend(B, q))
    refused(INVALID, lambda: fm.fm_paged_selftest_wait_timeout(B.c, 0))


def test_devices():
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    B = Batch([(1, 10)], 1, 1, 64, 16, TYPES["f16"], seed=34).create().fill_rows()
    q = B.queries()
    with torch.cuda.device(1):
        refused(INVALID, lambda: fm.fm_paged_attend(B.c, 0, B.b, q, torch.empty_like(q), workspace=torch.empty((B.b.workspace_bytes,), dtype=torch.uint8, device="cuda:0")))
        refused(INVALID, lambda: fm.fm_paged_synchronize(B.c))


@pytest.mark.parametrize("heads,seqs", [((16, 1, 128), 50), ((8, 2, 64), 64), ((4, 6, 256), 64)])
@pytest.mark.parametrize("new", [1, 2, 20])
def test_stages_are_read_before_they_are_refilled(heads, seqs, new):
    """Every SM's CTAs fetch at the memory's pace, so a stage is filled again as soon as it is given back: the same call gives
    the same bits however the warps run, and the oracle's values."""
    B = Batch([(1 + i % new, 1023 + i % 7) for i in range(seqs)], *heads, 64, TYPES["bf16"], seed=41).create().fill_rows()
    q = B.queries()
    first = torch.empty_like(q)
    fm.fm_paged_attend(B.c, 0, B.b, q, first)
    differs = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        out = torch.full_like(q, 7.0)
        fm.fm_paged_attend(B.c, 0, B.b, q, out)
        differs += (out != first).any()
    fm.fm_paged_synchronize(B.c)
    assert int(differs) == 0
    check_attend(B, q, first)
