"""The 4-bit KV cache (fm_kvq_*) through the C ABI against the fp64 oracle on the same rows.

Stored rows, evictions and weights that are moved are compared exactly.  Attention's tolerance, per output value, with
S = sum_j p_j |v_j| and A = scale max_j sum_d |q_d| K_jd, K_jd the largest |k_j| in d's group of 32:
  scores    f32 queries are f16 hi + lo (2^-22 of each term).  The codes enter as whole numbers n in 0 .. 15 and the f32 sum of a
            group starts at -8 sum q: its 32 products and the start value are exact or rounded once, and a partial sum is at
            most (15 + 8) / 8 of the group's part of A (a group's scale is an eighth of its largest value), so 33 additions err
            by 33 x 23 / 8 x 2^-24 A = 95 x 2^-24 A; the start value's own rounding 6 x 2^-24 A (a 32-term sum of 16-bit values
            by pairs); head_dim / 32 groups, the scale, log2(e) and the factor: (hd / 32 + 6) 2^-24 A; the reference's subtraction
            in the log2 domain 2^-22 x 1.45 A: delta <= (120 + hd / 32) 2^-24 A in all.  A probability is off by the factor
            e^(+-2 delta) with its sum's
            (f32 queries, and any with weights, take whole numbers n - 8 instead, in -8 .. 7: less.  Unsigned n are subnormals,
            by whose exponents the matrix instructions align a sum's terms: that costs f16 and bf16 outputs up to 6 bits of the
            24 in the worst case, which is not counted here -- their own rounding leaves more)
  exp2      2^-22 each, its sum's too
  P V       P' = p d (d the f16 scale) as f16.  bf16 outputs: p rounded, then the product, 2 x 2^-11 relative.  f16 outputs: p in two
            parts (2^-22), one rounding of the product 2^-11, of the second part's 2^-22.  f32 outputs: both parts of the product
            kept, 2^-21 in all.  Below f16's normal range a P' is off by 2^-25 absolute, times a code of at most 8, over 2^bias and a
            row sum of at least 1 (the reference is never above the largest score); bias = 7 - max(e, 0) with the largest scale
            vmax in [2^(e-1), 2^e) and e >= -6 (smaller scales are raised to that), so 8 2^-32 <= 2^-25 V a key for e < 0 and
            8 2^-25 2^(e-7) <= 2^-31 V above, V = 8 vmax the largest value the rows can hold.  (Against V, not S: where every key
            of weight has a 0 in a dimension, S falls below what the keys without weight round to.)
  sums      L products and the joins of parts in f32: (L + 64) 2^-24 S at most (a part's rescaling is a product more); f16 and
            bf16 outputs sum whole codes (up to 15 / 8 V a key) and take eight times the sum of P' (V) off at the end:
            (L + 64) 2^-24 x 3 V more
  output    half a step of its type
so |out - oracle| <= S (e^(2 delta) - 1 + 2^-20 + pv + (L + 64) 2^-23) + L floor V
[f16, bf16: + (L + 64) 2^-24 3 V] + eps / 2 |out|; a weight (f32, a sum of
R probabilities) is off by at most w (e^(2 delta) - 1 + 2^-20 + (L + R + 64) 2^-23)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import kvq as Q

pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_speculative_decoding_fm_gb300 import build
    build.build()


def ttype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def rows(rng, n, heads, hd, name, size=1.0):
    """Random rows as a CUDA tensor, and the values it holds."""
    import torch
    x = torch.from_numpy((rng.normal(size=(n, heads, hd)) * size).astype(np.float32)).to(ttype(name))
    return x.cuda(), x.double().numpy()


def check_out(got, want, mass, reach, hd, L, name, vals):
    import torch
    eps = torch.finfo(ttype(name)).eps
    delta = (120 + hd / 32) * 2.0 ** -24 * reach[..., None]
    pv = {"bf16": 2 * 2.0 ** -11, "f16": 2.0 ** -11 + 2.0 ** -21, "f32": 2.0 ** -21}[name]
    big = np.abs(vals).max(initial=0.0)
    floor = 2.0 ** -25 if big < 8.0 else 2.0 ** -31
    tol = mass * (np.expm1(2 * delta) + 2.0 ** -20 + pv + (L + 64) * 2.0 ** -23) + L * floor * big + eps / 2 * np.abs(want)
    tol += 0.0 if name == "f32" else (L + 64) * 2.0 ** -24 * 3 * big
    tol += 2.0 ** -25 if name == "f16" else 0.0    # f16 outputs below the normal range
    got = got.double().cpu().numpy()
    worst = np.max(np.abs(got - want) / np.maximum(tol, 1e-300)) if got.size else 0.0
    assert np.all(np.abs(got - want) <= tol), f"off by {worst:.2f} tolerances"


def check_weights(got, want, reach, hd, L, R):
    delta = (120 + hd / 32) * 2.0 ** -24 * reach.max() if reach.size else 0.0
    tol = np.abs(want) * (np.expm1(2 * delta) + 2.0 ** -20 + (L + R + 64) * 2.0 ** -23) + 1e-37
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


class Cache:
    """A cache and the values it should hold, per sequence [L, Hkv, hd]."""

    def __init__(self, n_seqs, hkv, hd, max_rows, n_layers=1):
        import block_speculative_decoding_fm_gb300 as fm
        self.fm, self.hkv, self.hd = fm, hkv, hd
        self.c = fm.fm_kvq_create(n_layers, n_seqs, hkv, hd, max_rows)
        self.k = {}
        self.v = {}

    def append(self, seqs, ns, starts, rng, name="f32", size=1.0, layer=0):
        import torch
        n = sum(ns)
        k, kv = rows(rng, n, self.hkv, self.hd, name, size)
        v, vv = rows(rng, n, self.hkv, self.hd, name, size)
        self.fm.fm_kvq_append(self.c, layer, seqs, k, v, ns, starts)
        at = 0
        for s, m, st in zip(seqs, ns, starts):
            for store, new in ((self.k, kv), (self.v, vv)):
                old = store.get((layer, s), np.zeros((0, self.hkv, self.hd)))[:st]
                store[layer, s] = np.concatenate([old, Q.stored(new[at:at + m])])
            at += m
        torch.cuda.synchronize()

    def read(self, s, name="f32", layer=0):
        import torch
        L = self.fm.fm_kvq_length(self.c, layer, s)
        k = torch.full((L, self.hkv, self.hd), 7.0, dtype=ttype(name), device="cuda")
        v = torch.full_like(k, 7.0)
        w = torch.full((1, self.hkv, max(1, L)), -1.0, device="cuda")
        self.fm.fm_kvq_read(self.c, layer, [s], [0], [L], k, v, w)
        self.fm.fm_kvq_synchronize(self.c)
        return k, v, w[0, :, :L].cpu().numpy()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
def test_append_read(hd, name):
    """Ragged appends at odd starts, rewinds, an empty one; the neighbours' rows stay."""
    import torch
    rng = np.random.default_rng(hd)
    c = Cache(3, 3, hd, 200)
    c.append([0, 2, 1], [130, 1, 64], [0, 0, 0], rng, name)
    c.append([2, 0], [31, 70], [1, 63], rng, name)          # sequence 0 is rewound into a tile
    c.append([1, 2], [0, 33], [17, 31], rng, name)          # no rows: only the length moves
    assert [c.fm.fm_kvq_length(c.c, 0, s) for s in range(3)] == [133, 17, 64]
    for s in range(3):
        for out in TYPES:
            k, v, w = c.read(s, out)
            for got, want in ((k, c.k[0, s]), (v, c.v[0, s])):
                assert torch.equal(got.cpu(), torch.from_numpy(want).to(ttype(out))), (s, out)
            assert np.all(w == 0)
    # a range in the middle, V alone
    v = torch.zeros((40, 3, hd), device="cuda")
    c.fm.fm_kvq_read(c.c, 0, [0], [50], [40], None, v)
    assert np.array_equal(v.cpu().numpy(), c.v[0, 0][50:90])


def test_append_extremes():
    """NaN, infinities, values past f16, borders between codes, scales that vanish: the stored values, bit for bit."""
    import torch
    rng = np.random.default_rng(9)
    x = rng.normal(size=(64, 1, 64)).astype(np.float32)
    x[0, 0, 5] = np.nan
    x[1, 0, 3], x[1, 0, 9] = np.inf, -np.inf
    x[2] *= 1e6
    x[3] *= 1e-8
    x[4] = 0.0
    x[5, 0, :32] = np.float32(0.5) * np.arange(-16, 16)          # d = 1: every second value on a border
    x[6, 0, :32] = -x[5, 0, :32]
    x[7, 0] = np.nan
    for r in range(8, 64):                                        # borders of random scales, and one step beside them
        d = np.float32(np.float16(rng.uniform(0.01, 3.0)))
        b = d * (rng.integers(-8, 8, size=64) + np.float32(0.5)).astype(np.float32)
        x[r, 0] = np.where(rng.random(64) < 0.4, b, np.nextafter(b, np.where(rng.random(64) < 0.5, np.inf, -np.inf).astype(np.float32)))
        x[r, 0, 0] = x[r, 0, 32] = -8 * d
    c = Cache(1, 1, 64, 64)
    t = torch.from_numpy(x).cuda()
    c.fm.fm_kvq_append(c.c, 0, [0], t, t, [64], [0])
    k, v, _ = c.read(0)
    want = Q.stored(x).astype(np.float32)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want)


def attend_case(c, seqs, T, group, name, rng, causal=False, first=0, decay=None, prior=None, scale=None, qsize=1.0):
    import torch
    H = c.hkv * group
    q, qv = rows(rng, sum(T), H, c.hd, name, qsize)
    out = torch.full_like(q, 9.0)
    Ls = [c.k[0, s].shape[0] for s in seqs]
    w = None if decay is None else torch.full((len(seqs), c.hkv, max(Ls) + 3), -5.0, device="cuda")
    c.fm.fm_kvq_attend(c.c, 0, seqs, q, T, out, scale=scale, causal=causal, first_row=first, decay=decay, weights=w)
    c.fm.fm_kvq_synchronize(c.c)
    at = 0
    for i, (s, t, L) in enumerate(zip(seqs, T, Ls)):
        want, ww, mass, reach = Q.attend(qv[at:at + t], c.k[0, s], c.v[0, s], c.hd ** -0.5 if scale is None else scale, causal, first)
        check_out(out[at:at + t], want, mass, reach, c.hd, L, name, c.v[0, s])
        if w is not None:
            got = w[i].cpu().numpy()
            if t:
                total = ww + (0.0 if prior is None else decay * prior[s])
                check_weights(got[:, :L].astype(np.float64), total, reach, c.hd, L, t * group)
                if prior is not None:
                    prior[s] = got[:, :L].astype(np.float64)
            else:
                assert np.all(got == -5.0)
            assert np.all(got[:, L:] == -5.0)    # behind the sequence's end: left as it was
        at += t
    return out


LENS = [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("hd,hkv,group", [(64, 2, 1), (64, 1, 5), (128, 2, 1), (128, 1, 8), (256, 1, 6), (256, 2, 1)])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("causal", [False, True])
def test_attend(hd, hkv, group, name, causal):
    """Every length around a tile's edges, no rows to many, rows that see nothing, with the weights."""
    rng = np.random.default_rng(hd + group + causal)
    c = Cache(len(LENS), hkv, hd, 310)
    ids = list(range(len(LENS)))
    # what the rows behind each end hold is large
    c.append(ids, [310] * len(ids), [0] * len(ids), rng, "f32", 1000.0)
    c.append(ids, LENS, [0] * len(ids), rng, name)
    for T in ([1] * len(ids), [2, 0, 5, 1, 17, 16, 3, 1, 0, 33, 8, 16]):
        attend_case(c, ids, T, group, name, rng, causal, decay=0.0)
    attend_case(c, ids[::-1], [3] * len(ids), group, name, rng, causal, first=40, decay=0.0)


@pytest.mark.parametrize("hd,hkv,group,T", [(128, 1, 1, 16), (256, 1, 6, 8), (64, 2, 2, 1)])
@pytest.mark.parametrize("name", TYPES)
def test_attend_split(hd, hkv, group, T, name):
    """A long sequence beside short ones: its keys are dealt to many CTAs and joined."""
    rng = np.random.default_rng(hd * 7 + T)
    c = Cache(3, hkv, hd, 9000)
    c.append([0, 1, 2], [9000, 5, 700], [0, 0, 0], rng, name)
    attend_case(c, [0, 1, 2], [T, T, T], group, name, rng, causal=True, decay=0.0, qsize=2.0)
    attend_case(c, [0], [T], group, name, rng, first=4321)
    for first in (8999, 9000, 2 ** 31 - 1):     # one row left, and none
        attend_case(c, [2, 0], [T, T], group, name, rng, first=first, decay=0.0)


def test_weights_accumulate():
    """Decay over calls; appended rows start at zero; rewound rows lose what they had."""
    rng = np.random.default_rng(4)
    c = Cache(2, 2, 64, 400)
    c.append([0, 1], [150, 90], [0, 0], rng)
    prior = {0: np.zeros((2, 150)), 1: np.zeros((2, 90))}
    for decay in (1.0, 0.5, 1.0):
        attend_case(c, [0, 1], [2, 3], 2, "f32", rng, True, decay=decay, prior=prior)
    c.append([0], [30], [140], rng)
    prior[0] = np.concatenate([prior[0][:, :140], np.zeros((2, 30))], 1)
    assert np.array_equal(c.read(0)[2], prior[0].astype(np.float32))
    attend_case(c, [1, 0], [1, 1], 2, "f32", rng, True, first=100, decay=0.25, prior=prior)
    before = c.read(0)[2]
    attend_case(c, [0], [4], 2, "f32", rng)                       # no decay: the weights are left alone
    assert np.array_equal(c.read(0)[2], before)


@pytest.mark.parametrize("size", [1e-6, 1e-3, 30.0, 6e4])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_attend_ranges(size, name):
    """Rows far from unit size: P times the V scale stays inside f16 either way."""
    rng = np.random.default_rng(11)
    c = Cache(1, 1, 128, 256)
    c.append([0], [200], [0], rng, "f32", size)
    attend_case(c, [0], [16], 1, name, rng, scale=0.1 / size)
    attend_case(c, [0], [16], 1, name, rng, scale=0.1, qsize=1.0 / size)


def test_attend_nan_and_peaks():
    """A NaN query row is NaN alone; one key far above the rest; a zero and a negative scale."""
    import torch
    rng = np.random.default_rng(12)
    c = Cache(1, 1, 64, 300)
    c.append([0], [300], [0], rng, "f32", 3.0)
    q, qv = rows(rng, 8, 1, 64, "f32")
    q[3, 0, 7] = float("nan")
    q[5] *= 200.0
    qv = q.double().cpu().numpy()
    for scale in (1.0, 0.0, -0.5):
        out = torch.zeros_like(q)
        c.fm.fm_kvq_attend(c.c, 0, [0], q, [8], out, scale=scale)
        ok = [0, 1, 2, 4, 5, 6, 7]
        assert bool(torch.isnan(out[3]).all())
        want, _, mass, reach = Q.attend(qv[ok], c.k[0, 0], c.v[0, 0], scale)
        check_out(out[ok], want, mass, reach, 64, 300, "f32", c.v[0, 0])


def test_strides():
    """Rows inside wider ones (a stacked q/k/v product), for every call."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    rng = np.random.default_rng(13)
    hd, hkv, H, n = 64, 2, 4, 70
    wide, val = rows(rng, n, H + 2 * hkv, hd, "f16")
    q, k, v = wide[:, :H], wide[:, H:H + hkv], wide[:, H + hkv:]
    c = fm.fm_kvq_create(1, 1, hkv, hd, n)
    fm.fm_kvq_append(c, 0, [0], k, v, [n], [0])
    outw = torch.full((5, 2 * H, hd), 3.0, dtype=torch.float16, device="cuda")
    fm.fm_kvq_attend(c, 0, [0], q[-5:], [5], outw[:, H:], causal=True)
    ks, vs = Q.stored(val[:, H:H + hkv]), Q.stored(val[:, H + hkv:])
    want, _, mass, reach = Q.attend(val[-5:, :H], ks, vs, hd ** -0.5, True)
    check_out(outw[:, H:], want, mass, reach, hd, n, "f16", vs)
    assert bool((outw[:, :H] == 3.0).all())
    back = torch.full((n, 3 * hkv, hd), 2.0, device="cuda")
    fm.fm_kvq_read(c, 0, [0], [0], [n], back[:, :hkv], back[:, 2 * hkv:])
    assert np.array_equal(back[:, :hkv].cpu().numpy(), ks) and np.array_equal(back[:, 2 * hkv:].cpu().numpy(), vs)
    assert bool((back[:, hkv:2 * hkv] == 2.0).all())
    fm.fm_kvq_destroy(c)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("keep,recent", [(0, 0), (1, 0), (1, 1), (64, 64), (100, 17), (333, 0), (2000, 10), (5000, 7)])
def test_evict(hd, in_place, keep, recent):
    """Ragged lengths below and above keep, ties, NaN, zero and negative weights: rows kept, values and weights exact;
    a source that is not the destination stays."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    rng = np.random.default_rng(keep + recent + hd)
    lens = [2500, 1, 0, keep, keep + 1, 777]
    lens = [min(x, 2600) for x in lens]
    n, hkv = len(lens), 2
    c = Cache(2 * n, hkv, hd, 5000)
    ids = list(range(n))
    to = ids if in_place else [2 * n - 1 - i for i in ids]
    c.append(ids, lens, [0] * n, rng)
    w = np.round(np.abs(rng.normal(size=(n, hkv, max(lens)))) * 4).astype(np.float32) / 4   # many ties
    w[0] = rng.permutation(w[0].size).reshape(w[0].shape)                                   # none
    w[5, 0, ::3], w[5, 0, 1::7], w[5, 1] = np.nan, -1.5, -0.0
    w[5, 1, 50:60] = 0.0
    fm.fm_kvq_set_weights(c.c, 0, ids, torch.from_numpy(w).cuda())
    kept = torch.full((n, hkv, keep), -7, dtype=torch.int32, device="cuda")
    fm.fm_kvq_evict(c.c, 0, ids, to, keep, recent, kept)
    fm.fm_kvq_synchronize(c.c)
    for i, L in enumerate(lens):
        left = min(keep, L)
        assert fm.fm_kvq_length(c.c, 0, to[i]) == left
        k, v, gw = c.read(to[i])
        for h in range(hkv):
            want = Q.kept_rows(w[i, h, :L], keep, recent)
            got = kept[i, h].cpu().numpy()
            assert np.array_equal(got[:left], want) and np.all(got[left:] == -7), (i, h)
            assert np.array_equal(k[:, h].cpu().numpy(), c.k[0, i][want, h])
            assert np.array_equal(v[:, h].cpu().numpy(), c.v[0, i][want, h])
            assert np.array_equal(gw[h], w[i, h, want], equal_nan=True)
        if not in_place:
            assert fm.fm_kvq_length(c.c, 0, i) == L
            k, v, gw = c.read(i)
            assert np.array_equal(k.cpu().numpy(), c.k[0, i]) and np.array_equal(v.cpu().numpy(), c.v[0, i])


def test_serving_run():
    """The calls as a server makes them, on a cache of two layers: a prompt, tokens that keep their weights, a branch, an
    eviction at the budget, and more tokens over what is left."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    rng = np.random.default_rng(21)
    hd, hkv, group, keep, recent = 128, 2, 4, 96, 32
    c = fm.fm_kvq_create(2, 3, hkv, hd, 256)
    ks, vs, ws = {}, {}, {}
    for layer in range(2):
        for s, n in ((0, 150), (1, 80)):
            k, kv = rows(rng, n, hkv, hd, "bf16")
            v, vv = rows(rng, n, hkv, hd, "bf16")
            fm.fm_kvq_append(c, layer, [s], k, v, [n], [0])
            ks[layer, s], vs[layer, s], ws[layer, s] = Q.stored(kv), Q.stored(vv), np.zeros((hkv, n))

    def token(layer, seqs):
        k, kv = rows(rng, len(seqs), hkv, hd, "bf16")
        v, vv = rows(rng, len(seqs), hkv, hd, "bf16")
        q, qv = rows(rng, len(seqs), hkv * group, hd, "bf16", 2.0)
        out = torch.empty_like(q)
        starts = [fm.fm_kvq_length(c, layer, s) for s in seqs]
        fm.fm_kvq_append(c, layer, seqs, k, v, [1] * len(seqs), starts)
        fm.fm_kvq_attend(c, layer, seqs, q, [1] * len(seqs), out, causal=True, decay=1.0)
        for i, s in enumerate(seqs):
            # (per head the rows differ after an eviction: each head's own store)
            ks[layer, s] = np.concatenate([ks[layer, s], Q.stored(kv[i:i + 1])])
            vs[layer, s] = np.concatenate([vs[layer, s], Q.stored(vv[i:i + 1])])
            want, w, mass, reach = Q.attend(qv[i:i + 1], ks[layer, s], vs[layer, s], hd ** -0.5, True)
            ws[layer, s] = np.concatenate([ws[layer, s], np.zeros((hkv, 1))], 1) + w
            check_out(out[i:i + 1], want, mass, reach, hd, ks[layer, s].shape[0], "bf16", vs[layer, s])

    for _ in range(3):
        for layer in range(2):
            token(layer, [1, 0])
    for layer in range(2):
        for src, dst in ((0, 2), (0, 0), (1, 1)):     # sequence 2 branches off 0 before 0 is brought down itself
            kept = torch.full((1, hkv, keep), -1, dtype=torch.int32, device="cuda")
            w = torch.zeros((1, hkv, 256), device="cuda")
            fm.fm_kvq_read(c, layer, [src], [0], [fm.fm_kvq_length(c, layer, src)], weights=w)
            held = w[0, :, :ks[layer, src].shape[0]].cpu().numpy()
            assert np.allclose(held, ws[layer, src], rtol=1e-3)
            fm.fm_kvq_evict(c, layer, [src], [dst], keep, recent, kept)
            left = min(keep, held.shape[1])
            want = [Q.kept_rows(held[h], keep, recent) for h in range(hkv)]
            assert np.array_equal(kept[0, :, :left].cpu().numpy(), np.stack(want))
            new = [np.stack([x[layer, src][want[h], h] for h in range(hkv)], 1) for x in (ks, vs)]
            ks[layer, dst], vs[layer, dst] = new
            ws[layer, dst] = np.stack([held[h][want[h]] for h in range(hkv)]).astype(np.float64)
    assert [fm.fm_kvq_length(c, 0, s) for s in range(3)] == [96, 83, 96]
    for _ in range(3):
        for layer in range(2):
            token(layer, [2, 0, 1])
    fm.fm_kvq_synchronize(c)


def test_streams_and_graph():
    """Calls from two streams come in order; a captured step replays."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    rng = np.random.default_rng(31)
    c = Cache(1, 1, 128, 4096)
    c.append([0], [4000], [0], rng, "bf16")
    q, qv = rows(rng, 16, 1, 128, "bf16")
    want, w, mass, reach = Q.attend(qv, c.k[0, 0], c.v[0, 0], 128 ** -0.5)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(s1 if i % 2 else s2):
            outs.append(torch.zeros_like(q))
            fm.fm_kvq_attend(c.c, 0, [0], q, [16], outs[-1], decay=0.0)
    torch.cuda.synchronize()
    for o in outs:
        check_out(o, want, mass, reach, 128, 4000, "bf16", c.v[0, 0])
        assert torch.equal(o, outs[0])            # the same call, the same bits
    out, wt = torch.zeros_like(q), torch.zeros((1, 1, 4000), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.fm_kvq_attend(c.c, 0, [0], q, [16], out, decay=1.0, weights=wt)
    fm.fm_kvq_attend(c.c, 0, [0], q, [16], outs[0], decay=0.0)
    torch.cuda.synchronize()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, outs[1])
    check_weights(wt[0].cpu().numpy().astype(np.float64), 4 * w, reach, 128, 4000, 64)


def test_refusals():
    """Every check of an argument comes before any launch, and leaves the lengths."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    c = fm.fm_kvq_create(1, 2, 2, 64, 40)
    x = torch.zeros((40, 2, 64), device="cuda")
    fm.fm_kvq_append(c, 0, [0], x, x, [10], [0])
    q = torch.zeros((4, 4, 64), device="cuda")
    o = torch.zeros_like(q)
    lib = fm.load_library()

    def bad(status, f, *a, **k):
        with pytest.raises(fm.FmError) as e:
            f(*a, **k)
        assert e.value.status == status, e.value

    inv = fm.FM_ERR_INVALID_ARG
    bad(inv, fm.fm_kvq_append, c, 1, [0], x, x, [1], [0])
    bad(inv, fm.fm_kvq_append, c, 0, [2], x, x, [1], [0])
    bad(inv, fm.fm_kvq_append, c, 0, [-1], x, x, [1], [0])
    bad(inv, fm.fm_kvq_append, c, 0, [1, 1], x, x, [1, 1], [0, 0])
    bad(inv, fm.fm_kvq_append, c, 0, [1], x, x, [-1], [0])
    bad(fm.FM_ERR_STATE, fm.fm_kvq_append, c, 0, [1], x, x, [1], [1])
    bad(fm.FM_ERR_STATE, fm.fm_kvq_append, c, 0, [0], x, x, [1], [-1])
    bad(fm.FM_ERR_CONTEXT_FULL, fm.fm_kvq_append, c, 0, [0], x, x, [31], [10])
    bad(inv, fm.fm_kvq_read, c, 0, [0], [5], [6], x, x)
    bad(inv, fm.fm_kvq_read, c, 0, [0], [-1], [6], x, x)
    bad(inv, fm.fm_kvq_read, c, 0, [0], [0], [6])
    bad(inv, fm.fm_kvq_attend, c, 0, [0], q[:, :3], [4], o[:, :3])           # 3 heads over 2
    bad(inv, fm.fm_kvq_attend, c, 0, [0], q, [-4], o)
    bad(inv, fm.fm_kvq_attend, c, 0, [0], q, [4], o, scale=float("nan"))
    bad(inv, fm.fm_kvq_attend, c, 0, [0], q, [4], o, first_row=-1)
    bad(inv, fm.fm_kvq_attend, c, 0, [0], q, [4], o, decay=float("inf"))
    bad(inv, fm.fm_kvq_attend, c, 0, [0, 0], q, [2, 2], o, decay=1.0)
    bad(inv, fm.fm_kvq_attend, c, 0, [0], q, [4], o, decay=1.0, weights=torch.zeros((1, 2, 9), device="cuda"))
    bad(inv, fm.fm_kvq_attend, c, 0, [0], q, [4], o, weights=torch.zeros((1, 2, 10), device="cuda"))
    bad(inv, fm.fm_kvq_set_weights, c, 0, [0], torch.zeros((1, 2, 9), device="cuda"))
    bad(inv, fm.fm_kvq_evict, c, 0, [0], [0], 4, 5)
    bad(inv, fm.fm_kvq_evict, c, 0, [0], [0], 41, 5)
    bad(inv, fm.fm_kvq_evict, c, 0, [0], [0], -1, 0)
    bad(inv, fm.fm_kvq_evict, c, 0, [0, 1], [1, 1], 4, 2)
    bad(inv, fm.fm_kvq_evict, c, 0, [0, 1], [1, 0], 4, 2)                    # read by one move, written by another
    flat = torch.zeros(4 * 256 + 8, device="cuda")
    shifted = flat[1:1 + 4 * 256].view(4, 4, 64)
    bad(inv, fm.fm_kvq_attend, c, 0, [0], shifted, [4], o)
    bad(inv, fm.fm_kvq_append, c, 0, [1], shifted[:, :2], shifted[:, :2], [4], [0])
    narrow = torch.zeros((4, 2 * 64 + 2), dtype=torch.float16, device="cuda")[:, :128].view(4, 2, 64)
    bad(inv, fm.fm_kvq_append, c, 0, [1], narrow, narrow, [4], [0])          # a row stride that is no whole 16 bytes
    assert lib.fm_kvq_append(c, 0, 1, None, None, None, None, None, 2, 128, None) == inv
    for f, a in ((fm.fm_kvq_attend, (c, 0, [0], q.double(), [4], o)), (fm.fm_kvq_attend, (c, 0, [0], q.cpu(), [4], o)),
                 (fm.fm_kvq_attend, (c, 0, [0], q, [5], o)), (fm.fm_kvq_attend, (c, 0, [0], q, [4], o.half())),
                 (fm.fm_kvq_append, (c, 0, [0], x, x.half(), [4], [0])), (fm.fm_kvq_append, (c, 0, [0], x, x, [4, 4], [0])),
                 (fm.fm_kvq_append, (c, 0, [0], x.transpose(1, 2), x, [4], [0])),
                 (fm.fm_kvq_evict, (c, 0, [0], [0], 4, 2, torch.zeros((1, 2, 5), dtype=torch.int32, device="cuda")))):
        with pytest.raises(ValueError):
            f(*a)
    assert fm.fm_kvq_length(c, 0, 0) == 10 and fm.fm_kvq_length(c, 0, 1) == 0
    with pytest.raises(fm.FmError):
        fm.fm_kvq_length(c, 0, 2)
    assert fm.fm_kvq_memory_bytes(c) > 0
    fm.fm_kvq_destroy(c)
