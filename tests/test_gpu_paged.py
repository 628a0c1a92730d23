"""The paged KV cache on the GPU against the fp64 oracle: attention of single tokens, blocks and chunks, grouped heads,
windows with sinks, ragged batches; writing with norms and rotation."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_speculative_decoding_fm_gb300 as fm
from oracle import paged as P
from paged_common import TYPES, Batch, check_attend, half_step

pytestmark = pytest.mark.gpu

# (new, past) rows of the sequences
TOKENS = [(1, 0), (1, 62), (1, 63), (1, 64), (0, 40), (1, 500), (1, 1)]
BLOCKS = [(16, 0), (3, 100), (16, 240), (5, 59), (1, 7)]
CHUNKS = [(17, 0), (130, 1), (64, 200), (0, 0), (128, 128), (1, 300), (257, 0)]


def attend(B, q, **kw):
    out = torch.full_like(q, 7.0)
    fm.fm_paged_attend(B.c, B.layer, B.b, q, out, **kw)
    fm.fm_paged_synchronize(B.c)
    return out


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(2, 1, 64), (1, 4, 64), (2, 1, 128), (1, 8, 128), (2, 6, 256), (1, 16, 256)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_tokens(t, heads, page):
    B = Batch(TOKENS, *heads, page, TYPES[t], seed=1).create().fill_rows()
    q = B.queries()
    check_attend(B, q, attend(B, q))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(2, 1, 64), (3, 1, 128), (2, 1, 256), (1, 5, 64), (2, 3, 256), (1, 7, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_blocks(t, heads, causal):
    B = Batch(BLOCKS, *heads, 32, TYPES[t], seed=2).create().fill_rows()
    q = B.queries()
    check_attend(B, q, attend(B, q, causal=causal), causal=causal)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(2, 1, 64), (1, 3, 64), (2, 1, 128), (1, 6, 128), (1, 1, 256), (1, 6, 256), (1, 128, 64)])
@pytest.mark.parametrize("page", [16, 128])
def test_chunks(t, heads, page):
    B = Batch(CHUNKS, *heads, page, TYPES[t], seed=3).create().fill_rows()
    q = B.queries()
    check_attend(B, q, attend(B, q))


@pytest.mark.parametrize("heads", [(2, 1, 64), (2, 1, 128), (1, 2, 256)])
def test_chunks_without_order(heads):
    B = Batch(CHUNKS, *heads, 64, TYPES["bf16"], seed=4).create().fill_rows()
    q = B.queries()
    check_attend(B, q, attend(B, q, causal=False), causal=False)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (40, 0), (64, 4), (100, 70), (128, 130), (2 ** 31 - 1, 0), (300, 2 ** 31 - 1)])
@pytest.mark.parametrize("heads", [(2, 1, 64), (1, 4, 128), (1, 3, 256)])
def test_window(window, sinks, heads):
    for seqs, page in ((TOKENS + [(1, 900)], 16), (BLOCKS + [(12, 700)], 64), (CHUNKS + [(140, 600)], 32)):
        B = Batch(seqs, *heads, page, TYPES["bf16"], seed=5).create().fill_rows()
        q = B.queries()
        check_attend(B, q, attend(B, q, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("heads,new,past", [((2, 2, 64), 1, 30000), ((1, 1, 128), 16, 20000), ((1, 8, 256), 2, 20001), ((1, 1, 64), 140, 9000),
                                            ((1, 2, 128), 70, 9100), ((1, 2, 256), 60, 8000)])
def test_split_keys(heads, new, past):
    """Few units over long sequences: each is cut between many CTAs and joined."""
    B = Batch([(new, past)], *heads, 128, TYPES["f16"], seed=6).create().fill_rows()
    q = B.queries()
    got = attend(B, q)
    check_attend(B, q, got)
    assert torch.equal(got, attend(B, q)), "the same call, other bits"


def test_many_sequences():
    """More sequences than a CTA has threads, some without rows."""
    rng = np.random.default_rng(7)
    seqs = [(int(rng.integers(0, 3)), int(rng.integers(0, 40))) for _ in range(700)]
    for heads in ((1, 2, 64), (1, 20, 64)):
        B = Batch(seqs, *heads, 16, TYPES["bf16"], seed=7).create().fill_rows()
        q = B.queries()
        check_attend(B, q, attend(B, q))


ROPES = [dict(rot=0), dict(rot=64, half=False, theta=1e4), dict(rot=64, half=True, theta=1e7), dict(rot=16, half=True, theta=5e5, gain=1.2),
         dict(rot=48, half=False, theta=1e4, scaling="linear", factor=4.0), dict(rot=32, half=True, theta=1e4, scaling="parts", factor=8.0, gain=1.2)]
KIND = {"none": fm.FM_ROPE_PLAIN, "linear": fm.FM_ROPE_LINEAR, "parts": fm.FM_ROPE_BY_PARTS}


def rope_args(r):
    if not r["rot"]:
        return {}, np.zeros(0)
    a = dict(scaling="none", factor=1.0, gain=1.0) | r
    f = P.frequencies(a["rot"], a["theta"], a["scaling"], a["factor"], 4096, 1.0, 32.0)
    return dict(rot_dims=a["rot"], layout=fm.FM_ROPE_HALF if a["half"] else fm.FM_ROPE_INTERLEAVED, theta=a["theta"], scaling=KIND[a["scaling"]],
                factor=a["factor"], original_rows=4096, low=1.0, high=32.0, gain=a["gain"]), f


def check_write(B, q, k, v, q_out, norms, freq, r, before):
    half, gain = r.get("half", False), r.get("gain", 1.0)
    pos = np.concatenate([np.arange(b, a + b) for a, b in B.seqs] + [np.zeros(0)])
    n = len(pos)
    e = half_step(B.t)
    want = {}
    for x, w, name in ((q, norms[0], "q"), (k, norms[1], "k")):
        y, reach = P.norm_rotate(x[:n].double().cpu().numpy(), None if w is None else w.cpu().numpy(), 1e-6, pos, freq, half, gain)
        want[name] = (y, e * np.abs(y) + 2e-6 * reach + torch.finfo(B.t).tiny * torch.finfo(B.t).eps)
    vv = v[:n].double().cpu().numpy()
    want["v"] = (vv, e * np.abs(vv) + torch.finfo(B.t).tiny * torch.finfo(B.t).eps)
    got = q_out[:n].double().cpu().numpy()
    assert (np.abs(got - want["q"][0]) <= want["q"][1]).all(), "q"
    first = 0
    written = torch.zeros(B.k_pool.shape[:4], dtype=torch.bool)
    for i, (a, b) in enumerate(B.seqs):
        for name, pool in (("k", B.k_pool), ("v", B.v_pool)):
            rows = B.rows(i, pool)[b:]
            y, tol = want[name]
            assert (np.abs(rows - y[first:first + a]) <= tol[first:first + a]).all(), name
        for j in range(b, a + b):
            written[B.layer, B.table_np[i, j // B.page], :, j % B.page] = True
        first += a
    for pool, old in zip((B.k_pool, B.v_pool), before):
        assert torch.equal(pool.cpu()[~written], old.cpu()[~written]), "rows that no call names"


@pytest.mark.parametrize("t,rows", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("heads", [(2, 2, 64), (1, 3, 128), (2, 1, 256)])
@pytest.mark.parametrize("r", range(len(ROPES)))
def test_write(t, rows, heads, r):
    r = ROPES[r]
    rope, freq = rope_args(r)
    B = Batch([(1, 5), (17, 30), (0, 9), (70, 0), (3, 100000)], *heads, 32, TYPES[t], seed=8, layers=3, layer=1, fill=3.0, pad=2).create(**rope)
    dt = torch.float32 if rows == "f32" else TYPES[t]
    x = torch.from_numpy(B.rng.normal(size=(B.total, B.heads + 2 * B.kv, B.hd)) * 2).to(dt).cuda()
    q, k, v = x[:, :B.heads], x[:, B.heads:B.heads + B.kv], x[:, B.heads + B.kv:]
    q_out = torch.full((B.total, B.heads, B.hd), 9.0, dtype=TYPES[t], device="cuda")
    before = B.k_pool.clone(), B.v_pool.clone()
    norms = [torch.from_numpy(1 + 0.1 * B.rng.normal(size=B.hd)).float().cuda() for _ in "qk"] if r["rot"] != 16 else [None, None]
    fm.fm_paged_write(B.c, B.layer, B.b, q, k, v, q_out, *norms)
    fm.fm_paged_synchronize(B.c)
    check_write(B, q, k, v, q_out, norms, freq, r, before)
    assert (q_out[-2:] == 9.0).all(), "rows behind the last sequence"


def test_write_many_tokens():
    """Large enough that a CTA takes several tokens, and sequences of one row beside long ones."""
    rope, freq = rope_args(ROPES[1])
    B = Batch([(1, 3)] * 40 + [(9000, 11)] + [(1, 0)] * 3, 1, 2, 64, 64, TYPES["bf16"], seed=9, fill=1.0).create(**rope)
    x = torch.from_numpy(B.rng.normal(size=(B.total, 4, 64))).to(B.t).cuda()
    q_out = torch.empty((B.total, 2, 64), dtype=B.t, device="cuda")
    before = B.k_pool.clone(), B.v_pool.clone()
    w = torch.ones(64, device="cuda")
    fm.fm_paged_write(B.c, 0, B.b, x[:, :2], x[:, 2:3], x[:, 3:], q_out, w, w)
    fm.fm_paged_synchronize(B.c)
    check_write(B, x[:, :2], x[:, 2:3], x[:, 3:], q_out, [w, w], freq, ROPES[1], before)


def test_far_positions():
    """Angles of positions near 2^30 (a turn is still resolved to 2^-25)."""
    f = P.frequencies(64, 1e4)
    page, past = 256, 2 ** 30 - 300
    k_pool = torch.zeros((1, 3, 1, page, 64), dtype=torch.float16, device="cuda")
    c = fm.fm_paged_create(k_pool, torch.zeros_like(k_pool), 1, rot_dims=64, theta=1e4)
    table = torch.zeros((1, 2 ** 22), dtype=torch.int32, device="cuda")
    table[0, past // page:past // page + 2] = torch.tensor([0, 1], device="cuda")
    b = fm.fm_paged_batch(c, torch.tensor([0, 300], dtype=torch.int32, device="cuda"), torch.tensor([2 ** 30], dtype=torch.int32, device="cuda"),
                          table, 300)
    x = torch.randn((300, 1, 64), device="cuda")
    out = torch.empty((300, 1, 64), dtype=torch.float16, device="cuda")
    fm.fm_paged_write(c, 0, b, x, x, x, out)
    fm.fm_paged_synchronize(c)
    y, reach = P.norm_rotate(x.double().cpu().numpy(), None, 0.0, np.arange(past, 2 ** 30), f, False)
    # (f_i is an f64: pos f_i is off by 2^30 2^-53, in the oracle as here)
    assert (np.abs(out.double().cpu().numpy() - y) <= half_step(torch.float16) * np.abs(y) + (2e-6 + 2.0 ** -21) * reach + 1e-7).all()
