"""The MTP head over a paged cache (fm_mtp_use_paged) against the oracle, with the head's own bars (h' within 2e-3, tokens exact
or excused by the margin): the rows' one rounding to f16 is 2^-11 of each, a fifth of the bar."""
from __future__ import annotations

import numpy as np
import pytest

import fm_synth as S
from gpu_common import REL_L2, rel_l2
from test_gpu_mtp import MtpPair, built, check_tokens, mid_config  # noqa: F401

pytestmark = pytest.mark.gpu


class PagedPair(MtpPair):
    def __init__(self, cfg, seed, pages=8, page=16, dtype="f16", window=0, sinks=0, **rope):
        import torch
        super().__init__(cfg.replace(kv_cap=1), seed)
        self.st = self.o.new_state(pages * page)
        t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        self.k, self.v = (torch.full((2, pages + 3, cfg.n_kv_heads, page, cfg.head_dim), float("nan"), dtype=t, device="cuda") for _ in "kv")
        args = dict(rot_dims=cfg.rot_dims, layout=self.fm.FM_ROPE_HALF, theta=cfg.theta, eps=cfg.eps) | rope
        self.c = self.fm.fm_paged_create(self.k, self.v, cfg.n_heads, **args)
        self.table = torch.from_numpy(np.random.default_rng(seed).permutation(pages + 3)[:pages].astype(np.int32)).cuda()
        self.fm.fm_mtp_use_paged(self.h, self.c, 1, self.table, window, sinks)

    def run(self, tokens, pos0, kv_lo=0, bar=REL_L2):
        """A pass; kv_lo: the oracle's first row."""
        import torch
        hn = S.gen_mtp_hidden(self.rng, len(tokens), self.cfg.hidden)
        hout = torch.zeros((len(tokens), self.cfg.hidden), dtype=torch.float32, device="cuda")
        drafts = torch.full((len(tokens),), -1, dtype=torch.int32, device="cuda")
        self.fm.fm_mtp_forward(self.h, torch.tensor(tokens, dtype=torch.int32, device="cuda"), torch.from_numpy(hn).cuda(), pos0, 0, hout,
                               drafts)
        self.fm.fm_paged_synchronize(self.c)
        ref = self.o.forward(self.st, self.o.embed(tokens), hn.astype(np.float64), pos0, kv_lo)
        assert rel_l2(hout.cpu().numpy(), ref.hout) < bar, rel_l2(hout.cpu().numpy(), ref.hout)
        if bar == REL_L2:
            lg = self.o.logits(ref.hout)
            check_tokens(drafts.cpu().numpy(), np.argmax(lg, axis=-1), lg)


@pytest.mark.parametrize("make", [S.mtp_micro_config, mid_config])
def test_passes(make):
    """Passes of several sizes and a rewind; pages in any order; the other layer's pages stay as they were."""
    p = PagedPair(make(), 1401)
    for tokens, pos in (([7, 8, 9, 10], 0), ([5, 17, 63], 4), ([11], 7), ([12, 13], 6), (list(range(100, 108)), 8), ([3], 16), ([4] * 8, 17)):
        p.run(tokens, pos)
    assert p.k[0].isnan().all() and p.v[0].isnan().all()
    assert p.fm.fm_mtp_last_launch_count(p.h) > 0
    p.close()


def test_bf16():
    """bf16 rows: q, k, v and the attention's rows are rounded to 2^-9 of each, four roundings of a branch of the stream."""
    p = PagedPair(mid_config(), 1402, dtype="bf16")
    for tokens, pos in (([7, 8, 9, 10], 0), ([5], 4), ([6, 7], 5)):
        p.run(tokens, pos, bar=4 * 2.0 ** -9)
    p.close()


def test_window():
    """A window over single-row passes: the oracle's first row moves with it."""
    p = PagedPair(S.mtp_micro_config(), 1403, window=5)
    for pos in range(12):
        p.run([20 + pos], pos, max(0, pos - 4))
    p.close()


def test_draft_chain():
    import torch
    cfg = S.mtp_micro_config()
    p = PagedPair(cfg, 1404)
    p.run([3, 4, 5, 6], 0)
    hn = S.gen_mtp_hidden(p.rng, 2, cfg.hidden)
    drafts = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    p.fm.fm_mtp_draft(p.h, torch.tensor([21, 22], dtype=torch.int32, device="cuda"), torch.from_numpy(hn).cuda(), 4, 0, 4, drafts)
    p.fm.fm_paged_synchronize(p.c)
    want, lg, _ = p.o.draft(p.st, [21, 22], hn.astype(np.float64), 4, 0, 4)
    check_tokens(drafts.cpu().numpy(), want, lg)
    p.close()


def test_own_cache_again():
    """Back to the head's own cache, to the 4-bit one and to the pages: each holds what it held."""
    import torch
    fm_cfg = S.mtp_micro_config()
    p = MtpPair(fm_cfg, 1405)
    p.forward([1, 2, 3], 0, 0)
    own = p.fm.fm_mtp_cache(p.h, 0, 3, np.empty((3, fm_cfg.n_kv_heads * fm_cfg.head_dim), np.float32))
    k, v = (torch.zeros((1, 4, fm_cfg.n_kv_heads, 16, fm_cfg.head_dim), dtype=torch.float16, device="cuda") for _ in "kv")
    c = p.fm.fm_paged_create(k, v, fm_cfg.n_heads, rot_dims=fm_cfg.rot_dims, layout=p.fm.FM_ROPE_HALF, theta=fm_cfg.theta, eps=fm_cfg.eps)
    table = torch.arange(4, dtype=torch.int32, device="cuda")
    p.fm.fm_mtp_use_paged(p.h, c, 0, table)
    t, hn = torch.tensor([9], dtype=torch.int32, device="cuda"), torch.from_numpy(S.gen_mtp_hidden(p.rng, 1, fm_cfg.hidden)).cuda()
    p.fm.fm_mtp_forward(p.h, t, hn, 0, 0)
    with pytest.raises(p.fm.FmError) as e:
        p.fm.fm_mtp_cache(p.h, 0, 1, np.empty((1, fm_cfg.n_kv_heads * fm_cfg.head_dim), np.float32))
    assert e.value.status == p.fm.FM_ERR_STATE
    kvq = p.fm.fm_kvq_create(1, 1, fm_cfg.n_kv_heads, fm_cfg.head_dim, 32)
    p.fm.fm_mtp_use_kvq(p.h, kvq)
    p.fm.fm_mtp_forward(p.h, t, hn, 0, 0)
    assert p.fm.fm_kvq_length(kvq, 0, 0) == 1
    p.fm.fm_mtp_use_paged(p.h, c, 0, table)
    p.fm.fm_mtp_forward(p.h, t, hn, 1, 0)
    assert p.fm.fm_kvq_length(kvq, 0, 0) == 1 and k[0, 0, :, 1].abs().sum() > 0
    p.fm.fm_mtp_use_paged(p.h, None)
    assert np.array_equal(own, p.fm.fm_mtp_cache(p.h, 0, 3, np.empty_like(own)))
    out, _, ref = p.forward([4], 3, 0)
    assert rel_l2(out, ref.hout) < REL_L2
    p.close()


def test_refusals():
    import torch
    cfg = S.mtp_micro_config()
    p = PagedPair(cfg, 1406, pages=2)
    fm = p.fm
    t, hn = torch.zeros((2,), dtype=torch.int32, device="cuda"), torch.zeros((2, cfg.hidden), device="cuda")

    def refused(status, call):
        with pytest.raises(fm.FmError) as e:
            call()
        assert e.value.status == status, str(e.value)

    before = p.k.clone()
    refused(fm.FM_ERR_CONTEXT_FULL, lambda: fm.fm_mtp_forward(p.h, t, hn, 31, 0))
    refused(fm.FM_ERR_CONTEXT_FULL, lambda: fm.fm_mtp_draft(p.h, t, hn, 29, 0, 3, torch.zeros((3,), dtype=torch.int32, device="cuda")))
    refused(fm.FM_ERR_UNSUPPORTED, lambda: fm.fm_mtp_forward(p.h, t, hn, 4, 1))
    assert torch.equal(before.nan_to_num(7), p.k.nan_to_num(7))
    bad = fm.FM_ERR_INVALID_ARG
    for kw in (dict(layer=2), dict(layer=-1), dict(window=-1), dict(sinks=3)):
        refused(bad, lambda: fm.fm_mtp_use_paged(p.h, p.c, **({"layer": 0, "table": p.table} | kw)))
    refused(bad, lambda: fm.fm_mtp_use_paged(p.h, p.c, 0, torch.zeros((0,), dtype=torch.int32, device="cuda")))
    good = dict(rot_dims=cfg.rot_dims, layout=fm.FM_ROPE_HALF, theta=cfg.theta, eps=cfg.eps)
    for change in (dict(rot_dims=16), dict(layout=fm.FM_ROPE_INTERLEAVED), dict(theta=5e4), dict(eps=1e-5)):
        c = fm.fm_paged_create(p.k, p.v, cfg.n_heads, **(good | change))
        refused(bad, lambda: fm.fm_mtp_use_paged(p.h, c, 0, p.table))
    refused(bad, lambda: fm.fm_mtp_use_paged(p.h, fm.fm_paged_create(p.k, p.v, 2 * cfg.n_heads, **good), 0, p.table))
    with pytest.raises(ValueError):
        fm.fm_mtp_use_paged(p.h, p.c, 0, p.table.long())
    p.close()
