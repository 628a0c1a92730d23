"""Slots of the 4-bit KV cache that held other rows before: what a call answers comes of the rows in view alone.  The rows
before are far larger (up to infinities), dropped by a rewind, an eviction, first_row or a shorter length; the answers are
a fresh slot's, bit for bit, and within test_gpu_kvq's tolerances of the oracle."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import kvq as Q
from test_gpu_kvq import TYPES, Cache, built, check_out, rows, ttype  # noqa: F401

pytestmark = pytest.mark.gpu

PASTS = [1e3, 1e6, np.inf]
T = 5


def past_rows(c, s, n, size, rng, start=0):
    """n rows of `size` behind `start` of sequence s, infinities among them where size is infinite."""
    import torch
    x = torch.from_numpy(rng.normal(size=(2, n, c.hkv, c.hd)).astype(np.float32) * (1e6 if np.isinf(size) else size))
    if np.isinf(size):
        x[:, ::7, :, ::5] = float("inf")
        x[:, 3::7, :, 1::5] = -float("inf")
    x = x.cuda()
    c.fm.fm_kvq_append(c.c, 0, [s], x[0], x[1], [n], [start])


def out_of(c, s, q, **k):
    import torch
    out = torch.full_like(q, 9.0)
    c.fm.fm_kvq_attend(c.c, 0, [s], q, [q.shape[0]], out, **k)
    c.fm.fm_kvq_synchronize(c.c)
    return out


def same_as_fresh(c, used, fresh, name, rng, **k):
    """Sequences `used` and `fresh` hold the same rows: the same bits, and the oracle's values."""
    import torch
    q, qv = rows(rng, T, 2 * c.hkv, c.hd, name, 2.0)
    got, want = out_of(c, used, q, **k), out_of(c, fresh, q, **k)
    assert bool(torch.isfinite(got).all())
    assert torch.equal(got, want)
    ks, vs = c.k[0, fresh], c.v[0, fresh]
    first = k.get("first_row", 0)
    ref, _, mass, reach = Q.attend(qv, ks, vs, c.hd ** -0.5, k.get("causal", False), first)
    check_out(got, ref, mass, reach, c.hd, len(ks), name, vs[first:])


def append_both(c, ids, n, start, size, rng):
    """The same n rows from `start` on in every sequence of ids."""
    import torch
    x = [torch.from_numpy((rng.normal(size=(n, c.hkv, c.hd)) * size).astype(np.float32)) for _ in "kv"]
    for s in ids:
        c.fm.fm_kvq_append(c.c, 0, [s], x[0].cuda(), x[1].cuda(), [n], [start])
        for store, y in ((c.k, x[0]), (c.v, x[1])):
            old = store.get((0, s), np.zeros((0, c.hkv, c.hd)))[:start]
            store[0, s] = np.concatenate([old, Q.stored(y.double().numpy())])


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("size", [1.0, 1e-3, 0.0])
@pytest.mark.parametrize("past", PASTS)
def test_restarted(hd, name, size, past):
    """Rewound to nothing and begun again."""
    rng = np.random.default_rng(hd)
    c = Cache(2, 2, hd, 400)
    past_rows(c, 0, 400, past, rng)
    append_both(c, [0, 1], 150, 0, size, rng)
    same_as_fresh(c, 0, 1, name, rng)
    same_as_fresh(c, 0, 1, name, rng, causal=True, first_row=33)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("past", PASTS)
def test_rejected_rows(hd, name, past):
    """A rewind into the middle: the rows that a draft added and lost."""
    rng = np.random.default_rng(hd + 1)
    c = Cache(2, 2, hd, 400)
    append_both(c, [0, 1], 90, 0, 1.0, rng)
    past_rows(c, 0, 200, past, rng, 90)
    append_both(c, [0, 1], 40, 90, 1.0, rng)
    same_as_fresh(c, 0, 1, name, rng, causal=True)
    c.fm.fm_kvq_append(c.c, 0, [0, 1], *([__import__("torch").zeros((0, 2, hd), device="cuda")] * 2), [0, 0], [70, 70])
    for s in (0, 1):
        c.k[0, s], c.v[0, s] = c.k[0, s][:70], c.v[0, s][:70]
    same_as_fresh(c, 0, 1, name, rng)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("size", [1.0, 1e-3, 0.0])
@pytest.mark.parametrize("past", PASTS)
def test_evicted_into(hd, name, size, past):
    """An eviction into a slot that held larger rows, and the rows kept of a source that has larger ones."""
    import torch
    rng = np.random.default_rng(hd + 2)
    c = Cache(4, 2, hd, 400)
    keep, recent = 150, 20
    past_rows(c, 1, 400, past, rng)
    append_both(c, [0], 300, 0, size, rng)
    w = rng.permutation(2 * 300).astype(np.float32).reshape(1, 2, 300)
    kept = [Q.kept_rows(w[0, h], keep, recent) for h in range(2)]
    # the same rows as values into a fresh slot: a stored row is stored again as it is
    for store in (c.k, c.v):
        store[0, 2] = np.stack([store[0, 0][kept[h], h] for h in range(2)], 1)
    k, v = (torch.from_numpy(store[0, 2].astype(np.float32)).cuda() for store in (c.k, c.v))
    c.fm.fm_kvq_append(c.c, 0, [2], k, v, [keep], [0])
    c.fm.fm_kvq_set_weights(c.c, 0, [0], torch.from_numpy(w).cuda())
    c.fm.fm_kvq_evict(c.c, 0, [0], [1], keep, recent)
    same_as_fresh(c, 1, 2, name, rng)
    # in place, from a slot whose lighter rows are the larger ones
    past_rows(c, 3, 400, past, rng)
    x = {}
    for key, store in (("k", c.k), ("v", c.v)):
        y = rng.normal(size=(300, 2, hd)) * past if np.isfinite(past) else np.full((300, 2, hd), np.inf)
        for h in range(2):
            y[kept[h], h] = store[0, 0][kept[h], h]
        x[key] = torch.from_numpy(y.astype(np.float32)).cuda()
    c.fm.fm_kvq_append(c.c, 0, [3], x["k"], x["v"], [300], [0])
    c.fm.fm_kvq_set_weights(c.c, 0, [3], torch.from_numpy(w).cuda())
    c.fm.fm_kvq_evict(c.c, 0, [3], [3], keep, recent)
    same_as_fresh(c, 3, 2, name, rng)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("past", PASTS)
def test_before_the_first_row(hd, name, past):
    """Large rows ahead of first_row, in its tile too."""
    rng = np.random.default_rng(hd + 3)
    c = Cache(2, 2, hd, 600)
    past_rows(c, 0, 300, past, rng)
    append_both(c, [1], 300, 0, 1.0, rng)
    c.k[0, 0], c.v[0, 0] = c.k[0, 1], c.v[0, 1]
    append_both(c, [0, 1], 250, 300, 1.0, rng)
    same_as_fresh(c, 0, 1, name, rng, first_row=300)


def check_large(c, name, rng, scale, causal=False):
    """Attention over sequence 0, whose outputs may pass f16's range: values from 65520 on are infinities there.  (Below 65000
    they are finite: a tolerance is under 1 % of the rows' mass, which is at most 2.8e5 with sizes up to 6e4.)"""
    import torch
    q, qv = rows(rng, T, 2 * c.hkv, c.hd, name)
    got = out_of(c, 0, q, scale=scale, causal=causal).double().cpu()
    want, _, mass, reach = Q.attend(qv, c.k[0, 0], c.v[0, 0], scale, causal)
    if name == "f16":
        over = torch.from_numpy(np.abs(want) > 65000)
        ref = torch.from_numpy(want)
        assert bool(((got * ref.sign())[over] > 64000).all())
        got = torch.where(over, ref, got)
    check_out(got, want, mass, reach, c.hd, len(c.k[0, 0]), name, c.v[0, 0])


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
def test_sizes_in_turn(hd, name):
    """One slot begun again with rows of every size, up and down."""
    rng = np.random.default_rng(hd + 4)
    c = Cache(2, 2, hd, 300)
    for size in (1e-6, 1.0, 6e4, 1e-3, 30.0, 1e-6, 6e4, 1.0):
        append_both(c, [0], 200, 0, size, rng)
        check_large(c, name, rng, 0.1 / size)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("jump", [1e2, 1e4, 6e4])
def test_sizes_in_one_sequence(hd, name, jump):
    """Values that grow and shrink along a sequence, over several tiles, seen together: the tolerance's V is the largest."""
    rng = np.random.default_rng(hd + 5)
    c = Cache(1, 2, hd, 1000)
    at = 0
    for n, size in ((150, 1e-3), (77, 1.0), (200, jump), (3, 1e-2), (400, 1.0), (20, jump)):
        append_both(c, [0], n, at, size, rng)
        at += n
    # (small queries: every row keeps some weight)
    for causal in (False, True):
        check_large(c, name, rng, 0.1 / jump, causal)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("big", [3e3, 8e4, 5e5])
def test_large_row_of_no_weight(hd, name, big):
    """A row in view with values up to what the cache can hold, whose key points away from every query, beside ordinary ones.
    P' of the keys that count (p from 1/4, a V scale from 2^-5) is 2^-14 at least in units of 2^(7 - 15) and kept to 2^-25: f32
    outputs within 2^-11; 16-bit ones within a step of their own."""
    import torch
    rng = np.random.default_rng(hd + 6)
    L, n, H = 1500, 16, 2
    k, v, q = rng.normal(size=(L, 1, hd)), rng.normal(size=(L, 1, hd)) * 0.5, rng.normal(size=(n, H, hd)) * 2
    k[:, 0, 0], q[:, :, 0] = 6.0, 30.0
    k[17, 0, 0], v[17] = -6.0, big * np.sign(v[17])
    dk, dv = (torch.from_numpy(x.astype(np.float32)).cuda() for x in (k, v))
    dq = torch.from_numpy(q.astype(np.float32)).to(ttype(name)).cuda()
    c = Cache(1, 1, hd, L)
    c.fm.fm_kvq_append(c.c, 0, [0], dk, dv, [L], [0])
    ks, vs = Q.stored(k.astype(np.float32)), Q.stored(v.astype(np.float32))
    want, w, _, _ = Q.attend_heads(dq.double().cpu().numpy(), ks, vs, hd ** -0.5)
    assert w[0, 17] < 1e-10
    got = out_of(c, 0, dq).double().cpu().numpy()
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert off <= {"f32": 2.0 ** -11, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[name], off
