"""The paged cache as programs lay things out: transposed rows, parts of larger batches and tables, shared pages, layers, many heads
and sequences, far positions, host threads, captures."""
from __future__ import annotations

import gc
import threading

import numpy as np
import pytest
import torch

import block_speculative_decoding_fm_gb300 as fm
from oracle import paged as P
from paged_common import TYPES, Batch, attend_bound, check_attend
from test_gpu_paged import BLOCKS, CHUNKS, TOKENS, attend

pytestmark = pytest.mark.gpu

KINDS = [(TOKENS, (2, 2, 64)), (BLOCKS, (2, 1, 128)), (CHUNKS, (2, 1, 128)), (CHUNKS, (1, 3, 64)), (CHUNKS, (1, 3, 256))]


@pytest.mark.parametrize("seqs,heads", KINDS)
def test_transposed_rows(seqs, heads):
    """Queries, outputs and rows to write laid out [heads, tokens, head_dim]."""
    B = Batch(seqs, *heads, 32, TYPES["bf16"], seed=71).create(rot_dims=32).fill_rows()
    q = B.queries()
    want = attend(B, q)
    turn = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)   # noqa: E731
    out = turn(torch.full_like(q, 7.0))
    fm.fm_paged_attend(B.c, 0, B.b, turn(q), out)
    fm.fm_paged_synchronize(B.c)
    assert torch.equal(out, want)
    k, v = (torch.randn((B.total, B.kv, B.hd), device="cuda").to(B.t) for _ in "kv")
    res = []
    for f in (lambda x: x, turn):
        B.k_pool.fill_(0.0), B.v_pool.fill_(0.0)
        q_out = f(torch.zeros_like(q))
        fm.fm_paged_write(B.c, 0, B.b, f(q), f(k), f(v), q_out)
        fm.fm_paged_synchronize(B.c)
        res.append((q_out.clone(), B.k_pool.clone(), B.v_pool.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("seqs,heads", KINDS)
def test_part_of_a_batch(seqs, heads):
    """Sequences 2 .. of a batch by views of its starts, lengths and a wider table: the other sequences' rows stay as they are."""
    B = Batch(seqs, *heads, 32, TYPES["f16"], seed=72).create().fill_rows()
    q = B.queries()
    want = attend(B, q)
    wide = torch.full((len(seqs), B.table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + B.table.shape[1]] = B.table
    b = fm.fm_paged_batch(B.c, B.starts[2:], B.len_dev[2:], wide[2:, 3:3 + B.table.shape[1]], B.total, max(B.n))
    out = torch.full_like(q, 7.0)
    fm.fm_paged_attend(B.c, 0, b, q, out)
    first = sum(B.n[:2])
    assert (out[:first] == 7.0).all()
    out[:first] = want[:first]
    check_attend(B, q, out)             # (units of another batch are cut elsewhere: not the same bits)
    q_out = torch.full_like(q, 7.0)
    fm.fm_paged_write(B.c, 0, b, q, None, None, q_out)
    fm.fm_paged_synchronize(B.c)
    assert torch.equal(q_out[first:], q[first:]) and (q_out[:first] == 7.0).all()


@pytest.mark.parametrize("heads,new", [((2, 1, 64), 1), ((1, 2, 128), 40), ((1, 2, 256), 40), ((1, 1, 64), 200)])
def test_shared_pages_and_layers(heads, new):
    """Sequences that begin with the same pages, in the second of three layers; the other layers' rows are NaN."""
    page, prefix = 16, 160
    B = Batch([(new, prefix + 40), (new, prefix + 7), (new, prefix)], *heads, page, TYPES["bf16"], seed=73, layers=3, layer=1).create().fill_rows()
    for i in (1, 2):
        B.table[i, :prefix // page] = B.table[0, :prefix // page]
        B.table_np[i, :prefix // page] = B.table_np[0, :prefix // page]
    q = B.queries()
    check_attend(B, q, attend(B, q))
    check_attend(B, q, attend(B, q, window=150, sinks=3), window=150, sinks=3)


def test_many_heads():
    """More heads than one CTA of the write takes, 128 of them to a KV head in the attention."""
    B = Batch([(1, 30), (3, 5)], 10, 128, 64, 16, TYPES["f16"], seed=74).create(rot_dims=64, layout=fm.FM_ROPE_HALF).fill_rows()
    x = torch.from_numpy(B.rng.normal(size=(B.total, B.heads + 2 * B.kv, 64))).half().cuda()
    q_out = torch.zeros((B.total, B.heads, 64), dtype=B.t, device="cuda")
    fm.fm_paged_write(B.c, 0, B.b, x[:, :B.heads], x[:, B.heads:B.heads + 10], x[:, B.heads + 10:], q_out)
    fm.fm_paged_synchronize(B.c)
    d, f = x.double().cpu().numpy(), P.frequencies(64, 1e4)
    pos = np.concatenate([np.arange(b, a + b) for a, b in B.seqs])
    for got, part in ((q_out.double().cpu().numpy(), d[:, :B.heads]),
                      (np.concatenate([B.rows(i, B.k_pool)[b:] for i, (_, b) in enumerate(B.seqs)]), d[:, B.heads:B.heads + 10])):
        y, reach = P.norm_rotate(part, None, 0.0, pos, f, True)
        assert (np.abs(got - y) <= 2.0 ** -11 * np.abs(y) + 2e-6 * reach + 1e-7).all()
    assert np.array_equal(np.concatenate([B.rows(i, B.v_pool)[b:] for i, (_, b) in enumerate(B.seqs)]), d[:, B.heads + 10:])
    check_attend(B, q_out, attend(B, q_out))
    few = fm.fm_paged_batch(B.c, B.starts, B.len_dev, B.table, B.total, 0)
    out = torch.full_like(q_out, 7.0)
    fm.fm_paged_attend(B.c, 0, few, q_out, out)
    fm.fm_paged_synchronize(B.c)
    check_attend(B, q_out, out)


@pytest.mark.parametrize("group", [1, 24])
def test_most_sequences(group):
    """65,536 sequences, one new row each."""
    n, hd, page = 65536, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    lengths = torch.randint(1, 17, (n,), generator=g, device="cuda", dtype=torch.int32)
    k_pool, v_pool = (torch.randn((1, n, 1, page, hd), generator=g, device="cuda").half() for _ in "kv")
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    c = fm.fm_paged_create(k_pool, v_pool, group)
    b = fm.fm_paged_batch(c, torch.arange(n + 1, dtype=torch.int32, device="cuda"), lengths, order[:, None].contiguous(), n, 1)
    q = torch.randn((n, group, hd), generator=g, device="cuda").half()
    out = torch.full_like(q, 7.0)
    fm.fm_paged_attend(c, 0, b, q, out)
    fm.fm_paged_synchronize(c)
    worst = 0.0
    for part in torch.arange(n, device="cuda").split(8192):
        k, v = (x[0, order[part].long(), 0].double() for x in (k_pool, v_pool))
        s = q[part].double() @ k.transpose(1, 2) * hd ** -0.5
        reach = (q[part].double().abs() @ k.abs().transpose(1, 2) * hd ** -0.5).amax(-1)
        s[(torch.arange(page, device="cuda")[None, None] >= lengths[part][:, None, None]).expand_as(s)] = float("-inf")
        p = s.softmax(-1)
        bound = attend_bound(torch.float16, (p @ v).cpu().numpy(), (p @ v.abs()).cpu().numpy(), reach.cpu().numpy(), page, float(v.abs().max()))
        worst = max(worst, float((np.abs((out[part].double() - p @ v).cpu().numpy()) / bound).max()))
    assert worst <= 1.0, worst
    k_rows = torch.randn((n, 1, hd), generator=g, device="cuda").half()
    fm.fm_paged_write(c, 0, b, None, k_rows, k_rows)
    fm.fm_paged_synchronize(c)
    at = (torch.arange(n, device="cuda"), lengths.long() - 1)
    for pool in (k_pool, v_pool):
        assert torch.equal(pool[0, order.long()][at[0], 0, at[1]], k_rows[:, 0])


@pytest.mark.parametrize("heads,new", [((1, 2, 64), 1), ((2, 1, 64), 200), ((1, 2, 128), 40), ((1, 1, 256), 30)])
def test_far_window(heads, new):
    """A window with sinks at the last of 2^30 rows: only the pages at both ends are there."""
    kv, group, hd = heads
    page, n, window, sinks = 256, 2 ** 30, 300, 5
    g = torch.Generator(device="cuda").manual_seed(6)
    k_pool, v_pool = (torch.randn((1, 5, kv, page, hd), generator=g, device="cuda").bfloat16() for _ in "kv")
    table = torch.full((1, n // page), -5, dtype=torch.int32, device="cuda")
    table[0, 0] = 3
    table[0, -3:] = torch.tensor([1, 4, 0], dtype=torch.int32, device="cuda")
    c = fm.fm_paged_create(k_pool, v_pool, kv * group)
    q = (torch.randn((new, kv * group, hd), generator=g, device="cuda") * 1.5).bfloat16()
    for length in (n, n - 100):
        b = fm.fm_paged_batch(c, torch.tensor([0, new], dtype=torch.int32, device="cuda"), torch.tensor([length], dtype=torch.int32, device="cuda"),
                              table, new)
        out = torch.full_like(q, 7.0)
        fm.fm_paged_attend(c, 0, b, q, out, window=window, sinks=sinks)
        fm.fm_paged_synchronize(c)
        d = q.double().cpu().numpy()
        ends = [x[0, [3, 1, 4, 0]].double().cpu().numpy().transpose(0, 2, 1, 3).reshape(4 * page, kv, hd) for x in (k_pool, v_pool)]
        for t in range(new):
            pos = length - new + t
            rows = list(range(sinks)) + [page + (j - (n - 3 * page)) for j in range(pos - window + 1, pos + 1)]
            k, v = (x[rows] for x in ends)
            want, mass, reach = P.attend(d[t:t + 1], k, v, hd ** -0.5)
            off = np.abs(out[t:t + 1].double().cpu().numpy() - want) / attend_bound(torch.bfloat16, want, mass, reach, len(rows), np.abs(v).max())
            assert off.max() <= 1.0, (t, off.max())


def test_host_threads():
    """Four threads write and attend over one cache, each in its own layer and stream."""
    heads, n, past = (2, 2, 64), 30, 500
    B = Batch([(n, past), (1, past)], *heads, 32, TYPES["f16"], seed=75, layers=4).create(rot_dims=32)
    rows = torch.randn((4, B.total, B.heads + 2 * B.kv, B.hd), device="cuda").half()
    B.k_pool.normal_(), B.v_pool.normal_()
    want, got, errors = [], [None] * 4, []

    def work(layer, stream):
        x = rows[layer]
        q, out = torch.zeros((B.total, B.heads, B.hd), dtype=B.t, device="cuda"), torch.zeros((B.total, B.heads, B.hd), dtype=B.t, device="cuda")
        fm.fm_paged_write(B.c, layer, B.b, x[:, :B.heads], x[:, B.heads:B.heads + B.kv], x[:, B.heads + B.kv:], q, stream=stream)
        fm.fm_paged_attend(B.c, layer, B.b, q, out, stream=stream)
        fm.fm_paged_synchronize(B.c, stream=stream)
        assert fm.fm_paged_last_launch_count(B.c) == 2
        return out

    for layer in range(4):
        want.append(work(layer, torch.cuda.current_stream()))

    def thread(layer):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(25):
                    got[layer] = work(layer, s)
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_collected_under_capture():
    """A cache that is collected while its thread captures leaves the capture as it is."""
    keep, gone = (Batch([(2, 50)], 1, 2, 64, 16, TYPES["f16"], seed=76).create().fill_rows() for _ in range(2))
    q = keep.queries()
    want = attend(keep, q)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.fm_paged_attend(keep.c, 0, keep.b, q, out)
        del gone
        gc.collect()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
