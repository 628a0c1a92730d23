"""Batches of a paged cache for the GPU tests: pools, tables and the error bounds of the two operators."""
from __future__ import annotations

import numpy as np
import torch

import block_speculative_decoding_fm_gb300 as fm
from oracle import paged as P

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(t):
    """A rounding to t is off by at most this, relative to the value."""
    return torch.finfo(t).eps / 2


class Batch:
    """Sequences of (new, past) rows in a pool of random pages in any order; unused rows and pages hold `fill`."""

    def __init__(self, seqs, kv_heads, group, hd, page, t, seed=0, layers=1, layer=0, fill=float("nan"), spare=2, cols=None, pad=0):
        rng = np.random.default_rng(seed)
        self.seqs, self.kv, self.group, self.hd, self.page, self.t, self.layer = seqs, kv_heads, group, hd, page, t, layer
        self.heads, self.rng = kv_heads * group, rng
        self.n = [a for a, _ in seqs]
        self.lengths = [max(0, a + b) for a, b in seqs]
        held = [-(-v // page) for v in self.lengths]
        cols = cols or max(held + [1])
        self.pages = sum(held) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        table = np.full((len(seqs), cols), -7, np.int32)   # (entries behind a sequence's end are not looked at)
        at = 0
        for i, v in enumerate(held):
            table[i, :v] = order[at:at + v]
            at += v
        self.table_np = table
        self.total = sum(self.n) + pad
        self.k_pool, self.v_pool = (torch.full((layers, self.pages, kv_heads, page, hd), fill, dtype=t, device="cuda") for _ in "kv")
        self.starts = torch.tensor(np.concatenate([[0], np.cumsum(self.n)]), dtype=torch.int32, device="cuda")
        self.len_dev = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.table = torch.from_numpy(table).cuda()

    def create(self, **rope):
        self.c = fm.fm_paged_create(self.k_pool, self.v_pool, self.heads, **rope)
        self.b = fm.fm_paged_batch(self.c, self.starts, self.len_dev, self.table, self.total, max(self.n + [0]))
        return self

    def rows(self, i, pool):
        """A sequence's rows [L, kv, hd] out of a pool, in 64 bits."""
        p = pool[self.layer].double().cpu().numpy()
        ids = self.table_np[i, :-(-self.lengths[i] // self.page)]
        x = p[ids].transpose(0, 2, 1, 3).reshape(-1, self.kv, self.hd)
        return x[:self.lengths[i]]

    def fill_rows(self, k_scale=1.0, v_scale=0.5):
        """Random rows in every sequence's places."""
        for pool, s in ((self.k_pool, k_scale), (self.v_pool, v_scale)):
            for i, n in enumerate(self.lengths):
                x = torch.from_numpy(self.rng.normal(size=(n, self.kv, self.hd)) * s).to(self.t).cuda()
                for j in range(0, n, self.page):
                    m = min(self.page, n - j)
                    pool[self.layer, int(self.table_np[i, j // self.page]), :, :m] = x[j:j + m].transpose(0, 1)
        return self

    def queries(self, scale=1.5):
        q = torch.from_numpy(self.rng.normal(size=(self.total, self.heads, self.hd)) * scale).to(self.t).cuda()
        return q


def attend_bound(t, out, mass, reach, keys, vmax):
    """Weights and output are rounded to t (half a step each); a score is a sum of products in f32 whose terms the matrix
    instructions align to the largest (2^-20 of the sum of their magnitudes covers it and exp2's 2^-22), and moves numerator
    and denominator; f16 weights below 2^-14 of the reference are off by up to 2^-25 a key."""
    e = half_step(t)
    bound = e * np.abs(out) + (e * (1 + e) + 2 * (reach[..., None] * 2.0 ** -20 + 2.0 ** -20)) * mass
    if t == torch.float16:
        bound = bound + keys * 2.0 ** -25 * vmax
    return bound + 1e-30


def check_attend(B, q, got, causal=True, window=0, sinks=0, scale=None):
    """The whole output against the oracle; rows of sequences with more new rows than rows are zeros."""
    worst, first = 0.0, 0
    qn, g = q.double().cpu().numpy(), got.double().cpu().numpy()
    for i, n in enumerate(B.n):
        if n:
            k, v = B.rows(i, B.k_pool), B.rows(i, B.v_pool)
            out, mass, reach = P.attend(qn[first:first + n], k, v, scale or B.hd ** -0.5, causal, window, sinks)
            vmax = np.abs(v).max() if len(v) else 0.0
            off = np.abs(g[first:first + n] - out) / attend_bound(B.t, out, mass, reach, len(k), vmax)
            assert np.isfinite(off).all(), f"sequence {i}: not finite"
            worst = max(worst, off.max(initial=0.0))
        first += n
    assert worst <= 1.0, f"{worst:.3f} of the bound"
    return worst
