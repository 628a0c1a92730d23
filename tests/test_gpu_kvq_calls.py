"""The 4-bit KV cache's calls (fm_kvq_*) beyond their ordinary sizes: units of many query rows over caches with work
enough for them, more sequences than one launch takes, captured calls, and the order of streams.  The helpers and
tolerances are test_gpu_kvq's."""
from __future__ import annotations

import gc

import numpy as np
import pytest

from oracle import kvq as Q
from test_gpu_kvq import TYPES, Cache, attend_case, built, check_out, check_weights, rows  # noqa: F401
from test_gpu_kvq import ttype

pytestmark = pytest.mark.gpu


def shared_rows(n_seqs, hkv, hd, lens, rng, name):
    """A cache whose sequences hold beginnings of the same rows."""
    import torch
    c = Cache(n_seqs, hkv, hd, max(lens))
    base = [rows(rng, max(lens), hkv, hd, name) for _ in range(2)]
    k, v = (torch.cat([b[0][:n] for n in lens]) for b in base)
    c.fm.fm_kvq_append(c.c, 0, list(range(n_seqs)), k, v, lens, [0] * n_seqs)
    ks, vs = (Q.stored(b[1]) for b in base)
    for s, n in enumerate(lens):
        c.k[0, s], c.v[0, s] = ks[:n], vs[:n]
    return c


@pytest.fixture
def by_products(monkeypatch):
    """attend_case's expectation by matrix products (the loops take minutes over many rows)."""
    monkeypatch.setattr(Q, "attend", Q.attend_heads)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("octets", [2, 3, 4])
@pytest.mark.usefixtures("by_products")
def test_wide_units(hd, name, octets):
    """48 sequences of 8 KV heads: a unit carries two, three or four octets of query rows (few rows go by one)."""
    rng = np.random.default_rng(hd + octets)
    n = 48
    lens = [520 + 13 * (i % 5) for i in range(n)]
    c = shared_rows(n, 8, hd, lens, rng, name)
    T = [4 * octets] * n                              # two query heads a KV head
    T[3], T[17], T[40] = 4 * octets - 1, 0, 1
    if octets == 4:
        T[9] = 35                                     # three tiles of 32, the last of 6
    attend_case(c, list(range(n)), T, 2, name, rng, causal=True, decay=0.0)
    attend_case(c, list(range(n))[::-1], T, 2, name, rng, first=130)


@pytest.mark.parametrize("hd", [64, 256])
def test_many_sequences(hd):
    """150 sequences a call, in launches of 64: every call, ragged, against each sequence by itself."""
    import torch
    rng = np.random.default_rng(41)
    n, hkv = 150, 2
    fm_lens = [int(x) for x in rng.integers(0, 140, n)]
    fm_lens[63], fm_lens[64], fm_lens[149] = 0, 139, 65
    c = Cache(n, hkv, hd, 140)
    ids = [int(x) for x in rng.permutation(n)]
    c.append(ids, [fm_lens[s] for s in ids], [0] * n, rng, "bf16")
    c.append(ids[::-1], [1] * n, [fm_lens[s] for s in ids[::-1]], rng, "bf16")
    attend_case(c, ids, [int(x) for x in rng.integers(0, 4, n)], 2, "f32", rng, causal=True, decay=0.0)
    # weights of the caller's, some alike; read back by range
    lens = [c.fm.fm_kvq_length(c.c, 0, s) for s in range(n)]
    assert lens == [x + 1 for x in fm_lens]
    w = rng.integers(0, 9, (n, hkv, 141)).astype(np.float32)
    c.fm.fm_kvq_set_weights(c.c, 0, list(range(n)), torch.from_numpy(w).cuda())
    at = [x // 3 for x in lens]
    take = [x - y for x, y in zip(lens, at)]
    k = torch.zeros((sum(take), hkv, hd), device="cuda")
    v, back = torch.zeros_like(k), torch.full((n, hkv, 150), -1.0, device="cuda")
    c.fm.fm_kvq_read(c.c, 0, ids, [at[s] for s in ids], [take[s] for s in ids], k, v, back)
    row = 0
    for i, s in enumerate(ids):
        assert np.array_equal(k[row:row + take[s]].cpu().numpy(), c.k[0, s][at[s]:]), s
        assert np.array_equal(v[row:row + take[s]].cpu().numpy(), c.v[0, s][at[s]:]), s
        assert np.array_equal(back[i, :, :take[s]].cpu().numpy(), w[s, :, at[s]:lens[s]]), s
        assert bool((back[i, :, take[s]:] == -1).all())
        row += take[s]
    # 70 in place and 40 into others that are given up
    src = ids[:70] + ids[70:110]
    dst = ids[:70] + ids[110:]
    keep, recent = 40, 7
    kept = torch.full((len(src), hkv, keep), -1, dtype=torch.int32, device="cuda")
    c.fm.fm_kvq_evict(c.c, 0, src, dst, keep, recent, kept)
    for i, (s, d) in enumerate(zip(src, dst)):
        left = min(keep, lens[s])
        assert c.fm.fm_kvq_length(c.c, 0, d) == left
        gk, gv, gw = c.read(d)
        for h in range(hkv):
            want = Q.kept_rows(w[s, h, :lens[s]], keep, recent)
            assert np.array_equal(kept[i, h, :left].cpu().numpy(), want), (s, h)
            assert np.array_equal(gk[:, h].cpu().numpy(), c.k[0, s][want, h])
            assert np.array_equal(gv[:, h].cpu().numpy(), c.v[0, s][want, h])
            assert np.array_equal(gw[h], w[s, h, want])
        assert bool((kept[i, :, left:] == -1).all())


def test_same_sequence_twice():
    """A call without weights may name a sequence more than once: each entry has its own query rows."""
    rng = np.random.default_rng(42)
    c = Cache(70, 2, 128, 300)
    c.append([0, 1], [300, 77], [0, 0], rng, "f16")
    attend_case(c, [0, 1, 0, 0, 1] * 14, [3, 1, 0, 5, 2] * 14, 2, "f16", rng, causal=True)


def test_source_twice():
    """One sequence read twice in a call, and branched into two others by one eviction; it stays as it is."""
    import torch
    rng = np.random.default_rng(50)
    c = Cache(4, 2, 64, 200)
    c.append([2, 3], [150, 20], [0, 0], rng, "f16")
    w = rng.normal(size=(1, 2, 150)).astype(np.float32)
    c.fm.fm_kvq_set_weights(c.c, 0, [2], torch.from_numpy(w).cuda())
    k = torch.zeros((40, 2, 64), device="cuda")
    c.fm.fm_kvq_read(c.c, 0, [2, 2, 3], [100, 90, 0], [10, 25, 5], k)
    want = np.concatenate([c.k[0, 2][100:110], c.k[0, 2][90:115], c.k[0, 3][:5]])
    assert np.array_equal(k.cpu().numpy(), want)
    c.fm.fm_kvq_evict(c.c, 0, [2, 2, 3], [0, 1, 3], 60, 9)
    assert [c.fm.fm_kvq_length(c.c, 0, s) for s in range(4)] == [60, 60, 150, 20]
    for d in (0, 1):
        gk, gv, gw = c.read(d)
        for h in range(2):
            rows_kept = Q.kept_rows(w[0, h], 60, 9)
            assert np.array_equal(gk[:, h].cpu().numpy(), c.k[0, 2][rows_kept, h])
            assert np.array_equal(gv[:, h].cpu().numpy(), c.v[0, 2][rows_kept, h])
            assert np.array_equal(gw[h], w[0, h, rows_kept])
    assert np.array_equal(c.read(2)[0].cpu().numpy(), c.k[0, 2]) and np.array_equal(c.read(3)[0].cpu().numpy(), c.k[0, 3])


def test_nothing_to_do():
    """Calls without rows: no query rows (weights counted or not), empty sequences, a keep of none, all rows kept."""
    import torch
    rng = np.random.default_rng(51)
    c = Cache(3, 2, 128, 100)
    c.append([0], [70], [0], rng, "bf16")
    none = torch.empty((0, 4, 128), device="cuda")
    before = c.read(0)
    w = torch.full((2, 2, 100), -3.0, device="cuda")
    for decay, weights in ((None, None), (0.0, w)):
        c.fm.fm_kvq_attend(c.c, 0, [0, 1], none, [0, 0], none.clone(), decay=decay, weights=weights)
    assert bool((w == -3).all())
    out = torch.full((3, 4, 128), 5.0, device="cuda")
    c.fm.fm_kvq_attend(c.c, 0, [1, 2], torch.ones_like(out), [1, 2], out, decay=1.0)
    assert bool((out == 0).all())
    kv = torch.empty((0, 2, 128), device="cuda")
    c.fm.fm_kvq_append(c.c, 0, [1, 2], kv, kv, [0, 0], [0, 0])
    c.fm.fm_kvq_read(c.c, 0, [1, 0], [0, 70], [0, 0], kv, kv)
    c.fm.fm_kvq_set_weights(c.c, 0, [1, 2], torch.empty((2, 2, 0), device="cuda"))
    c.fm.fm_kvq_evict(c.c, 0, [0, 1], [0, 1], 100, 0)
    for x, y in zip(before, c.read(0)):
        assert np.array_equal(np.asarray(x.cpu() if hasattr(x, "cpu") else x), np.asarray(y.cpu() if hasattr(y, "cpu") else y))
    c.fm.fm_kvq_evict(c.c, 0, [0], [2], 0, 0)
    assert [c.fm.fm_kvq_length(c.c, 0, s) for s in range(3)] == [70, 0, 0]
    c.fm.fm_kvq_synchronize(c.c)


@pytest.mark.parametrize("in_place", [True, False])
def test_captured_calls(in_place):
    """Append, attention with weights, eviction and read in one graph: replayed on the cache as it was at the capture it
    gives the eager calls' bits, also with new rows in its buffers."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    rng = np.random.default_rng(43)
    hd, hkv, n, keep, recent = 128, 2, 500, 200, 20

    def fresh():
        c = fm.fm_kvq_create(1, 2, hkv, hd, n + 8)
        fm.fm_kvq_append(c, 0, [0], k, v, [n], [0])
        return c

    def run(c, x):
        fm.fm_kvq_append(c, 0, [0], x["k"], x["v"], [8], [n])
        fm.fm_kvq_attend(c, 0, [0], x["q"], [8], x["out"], causal=True, decay=1.0, weights=x["w"])
        fm.fm_kvq_evict(c, 0, [0], [0 if in_place else 1], keep, recent, x["kept"])
        fm.fm_kvq_read(c, 0, [0 if in_place else 1], [0], [keep], x["ko"], x["vo"], x["wo"])

    def buffers(seed):
        r = np.random.default_rng(seed)
        x = {a: rows(r, 8, h, hd, "bf16")[0] for a, h in (("k", hkv), ("v", hkv), ("q", 2 * hkv))}
        x["out"] = torch.zeros_like(x["q"])
        x["w"] = torch.zeros((1, hkv, n + 8), device="cuda")
        x["kept"] = torch.zeros((1, hkv, keep), dtype=torch.int32, device="cuda")
        x["ko"] = torch.zeros((keep, hkv, hd), device="cuda")
        x["vo"] = torch.zeros_like(x["ko"])
        x["wo"] = torch.zeros((1, hkv, keep), device="cuda")
        return x

    k, v = rows(rng, n, hkv, hd, "bf16")[0], rows(rng, n, hkv, hd, "bf16")[0]
    wants = []
    for seed in (1, 2):
        c, x = fresh(), buffers(seed)
        run(c, x)
        fm.fm_kvq_synchronize(c)
        wants.append(x)
    c, x = fresh(), buffers(1)
    fm.fm_kvq_synchronize(c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c, x)
    assert fm.fm_kvq_length(c, 0, 0 if in_place else 1) == keep
    for want in wants:
        # the cache as it was: its rows again (which also puts their weights to 0)
        fm.fm_kvq_append(c, 0, [0], k, v, [n], [0])
        for a in ("k", "v", "q"):
            x[a].copy_(want[a])
        torch.cuda.synchronize()
        g.replay()
        fm.fm_kvq_synchronize(c)
        for a in want:
            assert torch.equal(x[a], want[a]), a


def test_two_graphs_share_a_cache():
    """Two captured calls of different shapes use one workspace: replayed in turn on a stream they do not disturb each
    other, nor an eager call between them."""
    import torch
    rng = np.random.default_rng(44)
    c = Cache(2, 2, 64, 5000)
    c.append([0, 1], [5000, 300], [0, 0], rng, "f16")
    cases, graphs = [], []
    for seqs, T in (([0], [16]), ([1, 0], [3, 2])):
        q, qv = rows(rng, sum(T), 4, 64, "f16")
        out = torch.zeros_like(q)
        c.fm.fm_kvq_attend(c.c, 0, seqs, q, T, out)
        torch.cuda.synchronize()
        cases.append((seqs, T, q, out, out.clone()))
        at = 0
        for s, t in zip(seqs, T):
            want, _, mass, reach = Q.attend(qv[at:at + t], c.k[0, s], c.v[0, s], 64 ** -0.5)
            check_out(out[at:at + t], want, mass, reach, 64, c.k[0, s].shape[0], "f16", c.v[0, s])
            at += t
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.fm.fm_kvq_attend(c.c, 0, seqs, q, T, out)
        graphs.append(g)
    for turn in range(6):
        for (_, _, _, out, _), g in zip(cases, graphs):
            out.zero_()
            g.replay()
        seqs, T, q, _, first = cases[turn % 2]
        eager = torch.zeros_like(q)
        c.fm.fm_kvq_attend(c.c, 0, seqs, q, T, eager)
        torch.cuda.synchronize()
        assert torch.equal(eager, first)
        for _, _, _, out, first in cases:
            assert torch.equal(out, first)


@pytest.mark.parametrize("shape", [(1024, 65536, 256, 256, 1 << 24), (1024, 65521, 241, 64, 1 << 24), (8, 4096, 8, 128, 1 << 24)])
def test_too_large(shape):
    """Sizes past the device's memory, and past what 64 bits count: refused, and the next cache is made as usual."""
    import block_speculative_decoding_fm_gb300 as fm
    with pytest.raises(fm.FmError) as e:
        fm.fm_kvq_create(*shape)
    assert e.value.status == fm.FM_ERR_OOM
    rng = np.random.default_rng(49)
    c = Cache(1, 1, 64, 64)
    c.append([0], [64], [0], rng)
    assert np.array_equal(c.read(0)[0].cpu().numpy(), c.k[0, 0])


def test_collected_under_capture():
    """A cache that is collected while its thread captures leaves the capture as it is."""
    import torch
    rng = np.random.default_rng(45)
    keep, gone = Cache(1, 1, 64, 64), Cache(1, 1, 64, 64)
    keep.append([0], [64], [0], rng)
    q, qv = rows(rng, 2, 1, 64, "f32")
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        keep.fm.fm_kvq_attend(keep.c, 0, [0], q, [2], out)
        del gone
        gc.collect()
    g.replay()
    torch.cuda.synchronize()
    want, _, mass, reach = Q.attend(qv, keep.k[0, 0], keep.v[0, 0], 64 ** -0.5)
    check_out(out, want, mass, reach, 64, 64, "f32", keep.v[0, 0])


def test_new_streams():
    """Streams that come and go between calls (a handle may be used again): each call still finds the last one's rows."""
    import torch
    rng = np.random.default_rng(46)
    c = Cache(1, 2, 128, 4100)
    c.append([0], [4000], [0], rng, "bf16")
    for i in range(12):
        k, kv = rows(rng, 8, 2, 128, "bf16")
        v, vv = rows(rng, 8, 2, 128, "bf16")
        q, qv = rows(rng, 8, 2, 128, "bf16")
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        for call in range(2):
            s = torch.cuda.ExternalStream(make_stream())
            with torch.cuda.stream(s):
                if call:
                    c.fm.fm_kvq_attend(c.c, 0, [0], q, [8], out, causal=True)
                else:
                    c.fm.fm_kvq_append(c.c, 0, [0], k, v, [8], [4000 + 8 * i])
            drop_stream(s.cuda_stream)      # (its work goes on)
        torch.cuda.synchronize()
        for store, new in ((c.k, kv), (c.v, vv)):
            store[0, 0] = np.concatenate([store[0, 0], Q.stored(new)])
        want, _, mass, reach = Q.attend(qv, c.k[0, 0], c.v[0, 0], 128 ** -0.5, True)
        check_out(out, want, mass, reach, 128, 4008 + 8 * i, "bf16", c.v[0, 0])


def test_offsets_past_32_bits():
    """A plane of 2^24 rows of 256 (4.8 GB), the longest a cache takes, and another behind it: every call at its end."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    rng = np.random.default_rng(48)
    hd, n, chunk = 256, 1 << 24, 1 << 20
    c = fm.fm_kvq_create(1, 2, 1, hd, n)
    filler = torch.randn((chunk, 1, hd), device="cuda", dtype=torch.bfloat16)
    tail = 333
    for at in range(0, n, chunk):
        fm.fm_kvq_append(c, 0, [0], filler, filler, [chunk], [at])
    k, kv = rows(rng, tail, 1, hd, "bf16")
    v, vv = rows(rng, tail, 1, hd, "bf16")
    fm.fm_kvq_append(c, 0, [0], k, v, [tail], [n - tail])
    assert fm.fm_kvq_length(c, 0, 0) == n
    ks, vs = Q.stored(kv), Q.stored(vv)
    back = [torch.zeros((tail, 1, hd), device="cuda") for _ in range(2)]
    fm.fm_kvq_read(c, 0, [0], [n - tail], [tail], *back)
    assert np.array_equal(back[0].cpu().numpy(), ks) and np.array_equal(back[1].cpu().numpy(), vs)
    w = torch.zeros((1, 1, n), device="cuda")
    for T, name in ((1, "bf16"), (9, "f32")):
        q, qv = rows(rng, T, 6, hd, name)
        out = torch.zeros_like(q)
        fm.fm_kvq_attend(c, 0, [0], q, [T], out, causal=True, first_row=n - tail, decay=0.0, weights=w)
        want, ww, mass, reach = Q.attend(qv, ks, vs, hd ** -0.5, True)
        check_out(out, want, mass, reach, hd, tail, name, vs)
        check_weights(w[0, :, n - tail:].cpu().numpy().astype(np.float64), ww, reach, hd, tail, 6 * T)
        assert float(w[0, 0, :n - tail].abs().max()) == 0.0
    # all rows: the filler is one chunk over and over, and a query of zeros weighs every row alike
    out = torch.zeros((1, 6, hd), device="cuda")
    fm.fm_kvq_attend(c, 0, [0], out.clone(), [1], out)
    full = [torch.zeros((chunk, 1, hd), device="cuda") for _ in range(2)]
    fm.fm_kvq_read(c, 0, [0], [0], [chunk], *full)
    f = full[1][:, 0].double()
    mean = (f.sum(0) * (n // chunk) - f[chunk - tail:].sum(0) + torch.from_numpy(vs[:, 0]).cuda().sum(0)) / n
    # (equal probabilities: a sum of n / 304 rows of up to 4 in f32 a CTA, over n: n / 304 x 2^-24 x the mean |v| of 0.8)
    assert float((out[0].double() - mean).abs().max()) <= n / 304 * 2.0 ** -24 * 0.8
    # eviction into the plane behind: distinct weights, whose largest lie anywhere
    order = torch.randperm(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    fm.fm_kvq_set_weights(c, 0, [0], order.float()[None, None])
    keep, recent = 1000, 10
    kept = torch.zeros((1, 1, keep), dtype=torch.int32, device="cuda")
    for dst in (1, 0):
        fm.fm_kvq_evict(c, 0, [0], [dst], keep, recent, kept)
        top = torch.topk(order[:n - recent], keep - recent).indices.sort().values
        want = torch.cat([top, torch.arange(n - recent, n, device="cuda")])
        assert torch.equal(kept[0, 0].long(), want)
        got = [torch.zeros((keep, 1, hd), device="cuda") for _ in range(2)]
        weights = torch.zeros((1, 1, keep), device="cuda")
        fm.fm_kvq_read(c, 0, [dst], [0], [keep], *got, weights)
        assert torch.equal(weights[0, 0], order[want].float())
        src = want % chunk
        for x, y, z in zip(got, full, (ks, vs)):
            end = torch.from_numpy(z.astype(np.float32)).cuda()
            ref = torch.where((want >= n - tail)[:, None, None], end[(want - (n - tail)).clamp(min=0)], y[src])
            assert torch.equal(x, ref)
    fm.fm_kvq_destroy(c)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_query_range(name):
    """Queries up to 2^97 (and tiny ones) with a scale that brings the scores back; far beyond, and infinite: NaN, that
    row's alone."""
    import torch
    rng = np.random.default_rng(47)
    c = Cache(1, 1, 64, 200)
    c.append([0], [200], [0], rng, "f16")
    for e in (-100, -60, 60, 96):
        q, qv = rows(rng, 4, 1, 64, name)
        q = q.clamp(-1.9, 1.9) * 2.0 ** e
        qv = q.double().cpu().numpy()
        bad = q.clone()
        bad[2, 0, 5] = float("inf") if e < 0 else 2.0 ** 110
        bad[3, 0, 60] = -bad[2, 0, 5]
        for x, ok in ((q, [0, 1, 2, 3]), (bad, [0, 1])):
            out = torch.zeros_like(x)
            c.fm.fm_kvq_attend(c.c, 0, [0], x, [4], out, scale=2.0 ** -e / 8)
            want, _, mass, reach = Q.attend(qv[ok], c.k[0, 0], c.v[0, 0], 2.0 ** -e / 8)
            check_out(out[ok], want, mass, reach, 64, 200, name, c.v[0, 0])
            assert len(ok) == 4 or bool(torch.isnan(out[2:]).all())


def test_misaligned_words():
    """Pointers to weights and kept rows that are no whole words are refused, and nothing moves."""
    import ctypes
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    c = fm.fm_kvq_create(1, 1, 1, 64, 40)
    x = torch.ones((30, 1, 64), device="cuda")
    fm.fm_kvq_append(c, 0, [0], x, x, [30], [0])
    lib = fm.load_library()
    room = torch.zeros(200, device="cuda")
    one = (ctypes.c_int32 * 1)
    s, n, zero = one(0), one(30), one(0)
    q, o = torch.ones((1, 1, 64), device="cuda"), torch.zeros((1, 1, 64), device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for off in (1, 2, 3):
        p = ctypes.c_void_p(room.data_ptr() + off)
        assert lib.fm_kvq_read(c, 0, 1, s, zero, n, None, None, fm.FM_DTYPE_F32, 64, p, 40, stream) == fm.FM_ERR_INVALID_ARG
        assert lib.fm_kvq_set_weights(c, 0, 1, s, p, 40, stream) == fm.FM_ERR_INVALID_ARG
        assert lib.fm_kvq_attend(c, 0, 1, s, one(1), q.data_ptr(), fm.FM_DTYPE_F32, 1, 64, 0.125, 0, 0, o.data_ptr(), 64, 1.0, p,
                                 40, stream) == fm.FM_ERR_INVALID_ARG
        assert lib.fm_kvq_evict(c, 0, 1, s, s, 10, 2, p, stream) == fm.FM_ERR_INVALID_ARG
        assert b"misaligned" in lib.fm_kvq_last_error(c)
    fm.fm_kvq_synchronize(c)
    assert fm.fm_kvq_length(c, 0, 0) == 30 and not bool(room.any()) and not bool(o.any())


def test_window_over_a_long_cache():
    """65,536 query rows of 8 heads over the last rows of 2^24: a call goes by the rows that it sees, not by those before
    them."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    rng = np.random.default_rng(51)
    hd, n, chunk, tail, T, H = 64, 1 << 24, 1 << 21, 200, 1 << 16, 8
    c = fm.fm_kvq_create(1, 1, 1, hd, n)
    filler = torch.ones((chunk, 1, hd), device="cuda", dtype=torch.bfloat16)
    for at in range(0, n, chunk):
        fm.fm_kvq_append(c, 0, [0], filler, filler, [chunk], [at])
    k, kv = rows(rng, tail, 1, hd, "bf16")
    v, vv = rows(rng, tail, 1, hd, "bf16")
    fm.fm_kvq_append(c, 0, [0], k, v, [tail], [n - tail])
    ks, vs = Q.stored(kv), Q.stored(vv)
    q = torch.randn((T, H, hd), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(torch.bfloat16)
    out = torch.full_like(q, 9.0)
    fm.fm_kvq_attend(c, 0, [0], q, [T], out, first_row=n - tail)
    fm.fm_kvq_synchronize(c)
    at = [0, 1, 31, 32, 4095, T // 2, T - 1]
    want, _, mass, reach = Q.attend_heads(q[at].double().cpu().numpy(), ks, vs, hd ** -0.5)
    check_out(out[at], want, mass, reach, hd, tail, "bf16", vs)
    fm.fm_kvq_destroy(c)


@pytest.mark.parametrize("nkv,group", [(1, 16), (2, 8)])
def test_most_query_rows(nkv, group):
    """2^15 units of 32 rows in one call, the most it takes, with the weights; one head more, one row more and one more head
    a KV head than may be are refused, and nothing is written."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    rng = np.random.default_rng(52)
    hd, n, T = 64, 100, 1 << 16
    c = Cache(1, nkv, hd, n)
    c.append([0], [n], [0], rng, "bf16")
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn((T, nkv * group, hd), device="cuda", generator=g).to(torch.bfloat16)
    out, w = torch.full_like(q, 9.0), torch.full((1, nkv, n), -1.0, device="cuda")
    fm.fm_kvq_attend(c.c, 0, [0], q, [T], out, decay=0.0, weights=w)
    fm.fm_kvq_synchronize(c.c)
    at = [0, 1, 4095, T // 2 + 1, T - 1]
    want, _, mass, reach = Q.attend_heads(q[at].double().cpu().numpy(), c.k[0, 0], c.v[0, 0], hd ** -0.5)
    check_out(out[at], want, mass, reach, hd, n, "bf16", c.v[0, 0])
    for h in range(nkv):
        k = torch.from_numpy(c.k[0, 0][:, h]).cuda()
        p = torch.zeros(n, dtype=torch.float64, device="cuda")
        for x in q[:, h * group:(h + 1) * group].split(T // 8):
            p += torch.softmax(x.double().reshape(-1, hd) @ k.T * hd ** -0.5, -1).sum(0)
        # (a sum in f32 of 2^15 tiles' parts: 2^15 roundings of 2^-24 of the sum so far, 2^-9 if all went one way; they do not,
        # which leaves room for the probabilities' own errors)
        assert float((w[0, h].double() / p - 1).abs().max()) < 2.0 ** -9

    def bad(status, q, n_rows):
        o = torch.full_like(q, 9.0)
        with pytest.raises(fm.FmError) as e:
            fm.fm_kvq_attend(c.c, 0, [0], q, [n_rows], o)
        assert e.value.status == status
        torch.cuda.synchronize()
        assert bool((o == 9.0).all())

    bad(fm.FM_ERR_UNSUPPORTED, torch.zeros((T, nkv * (group + 1), hd), dtype=torch.float16, device="cuda"), T)
    bad(fm.FM_ERR_INVALID_ARG, torch.zeros((T + 1, nkv, hd), dtype=torch.float16, device="cuda"), T + 1)
    bad(fm.FM_ERR_INVALID_ARG, torch.zeros((1, nkv * 1025, hd), dtype=torch.float16, device="cuda"), 1)
    many = torch.randn((3, nkv * 1024, hd), device="cuda", generator=g).to(torch.float16)
    out = torch.zeros_like(many)
    fm.fm_kvq_attend(c.c, 0, [0], many, [3], out, causal=True)
    want, _, mass, reach = Q.attend_heads(many.double().cpu().numpy(), c.k[0, 0], c.v[0, 0], hd ** -0.5, True)
    check_out(out, want, mass, reach, hd, n, "f16", c.v[0, 0])


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("big", [20.0, 400.0, 2000.0])
def test_outlier_channel(hd, name, big):
    """A channel that gives every score the same large part: what differs between the keys stays, with weights and without.
    The scores' own tolerance is large here (reach 1,000 and more), so the outputs are also held to what f32 scores lose
    by a plain sum of hd products of that size: each of its hd roundings 2^-25 reach off, sqrt(hd) of them together, three
    such deviations."""
    import torch
    rng = np.random.default_rng(53)
    L, T = 700, 16
    k = rng.normal(size=(L, 1, hd))
    k[:, 0, 5] = 8.0
    q = rng.normal(size=(T, 1, hd)) * 2
    q[:, 0, 5] = big * np.sign(rng.normal(size=T))
    k, q, v = (torch.from_numpy(x.astype(np.float32)).to(ttype(name)).cuda() for x in (k, q, rng.normal(size=(L, 1, hd))))
    c = Cache(1, 1, hd, L)
    c.fm.fm_kvq_append(c.c, 0, [0], k, v, [L], [0])
    ks, vs = (Q.stored(x.double().cpu().numpy()) for x in (k, v))
    want, _, mass, reach = Q.attend_heads(q.double().cpu().numpy(), ks, vs, hd ** -0.5)
    for decay in (None, 0.0):
        out = torch.zeros_like(q)
        c.fm.fm_kvq_attend(c.c, 0, [0], q, [T], out, decay=decay)
        check_out(out, want, mass, reach, hd, L, name, vs)
        off = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want)
        step = torch.finfo(out.dtype).eps / 2
        p = {"f32": 2.0 ** -21, "f16": 2.0 ** -11, "bf16": 2.0 ** -10}[name]
        assert off <= step + p + 3 * 2.0 ** -25 * hd ** 0.5 * reach.max() * 2 ** 0.5, off


def test_outputs_over_queries():
    """The queries' own rows as the outputs' are refused: other CTAs, and the weights' pass, still read them."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    c = fm.fm_kvq_create(1, 1, 1, 64, 40)
    x = torch.ones((30, 1, 64), device="cuda")
    fm.fm_kvq_append(c, 0, [0], x, x, [30], [0])
    q = torch.ones((2, 1, 64), device="cuda")
    with pytest.raises(fm.FmError) as e:
        fm.fm_kvq_attend(c, 0, [0], q, [2], q, decay=1.0)
    assert e.value.status == fm.FM_ERR_INVALID_ARG
    fm.fm_kvq_attend(c, 0, [0], q, [0], q)               # no rows: nothing to do
    fm.fm_kvq_synchronize(c)
    assert bool((q == 1).all())
    w = torch.full((1, 1, 30), -1.0, device="cuda")
    fm.fm_kvq_read(c, 0, [0], [0], [30], weights=w)
    assert bool((w == 0).all())


def runtime():
    import ctypes
    import glob
    import os
    import torch
    for p in ("libcudart.so.13", "libcudart.so", os.path.join(os.path.dirname(torch.__file__), "lib", "libcudart.so.13"),
              *glob.glob("/usr/local/cuda/lib64/libcudart.so*")):
        try:
            return ctypes.CDLL(p)
        except OSError:
            continue
    pytest.skip("no CUDA runtime library by name")


def make_stream():
    import ctypes
    s = ctypes.c_void_p()
    assert runtime().cudaStreamCreateWithFlags(ctypes.byref(s), 1) == 0
    return s.value


def drop_stream(handle):
    import ctypes
    assert runtime().cudaStreamDestroy(ctypes.c_void_p(handle)) == 0
