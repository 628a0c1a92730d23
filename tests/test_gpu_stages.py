"""Rings of stages in shared memory: a stage that a warp gives back is filled again at once, so its reads of it have to be done.
Where they are not, a call's bits go by how the warps run."""
from __future__ import annotations

import numpy as np
import pytest

import fm_synth as S
from gpu_common import REL_L2, Pair, rel_l2, tokens_match
from oracle import kvq as Q
from test_gpu_kvq import TYPES, built, check_out, rows  # noqa: F401
from test_gpu_kvq_calls import shared_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,hkv,group,T", [(64, 8, 2, 4), (128, 16, 1, 16), (256, 4, 6, 1), (256, 4, 6, 8)])
@pytest.mark.parametrize("name", TYPES)
def test_kvq_attention(hd, hkv, group, T, name):
    """32 sequences of the 4-bit cache, as fast as memory delivers them: the same call, the same bits, and the oracle's values."""
    import torch
    rng = np.random.default_rng(61)
    lens = [2017 + 13 * i for i in range(32)]
    c = shared_rows(32, hkv, hd, lens, rng, name)
    q, qv = rows(rng, 32 * T, hkv * group, hd, name)
    first = torch.full_like(q, 9.0)
    c.fm.fm_kvq_attend(c.c, 0, list(range(32)), q, [T] * 32, first)
    differs = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(50):
        out = torch.full_like(q, 7.0)
        c.fm.fm_kvq_attend(c.c, 0, list(range(32)), q, [T] * 32, out)
        differs += (out != first).any()
    c.fm.fm_kvq_synchronize(c.c)
    assert int(differs) == 0
    for s in (0, 17, 31):
        want, _, mass, reach = Q.attend_heads(qv[s * T:(s + 1) * T], c.k[0, s], c.v[0, s], hd ** -0.5)
        check_out(first[s * T:(s + 1) * T], want, mass, reach, hd, lens[s], name, c.v[0, s])
    c.fm.fm_kvq_destroy(c.c)


@pytest.mark.parametrize("target_dim", [384, 512, 2560])
def test_lm_head(target_dim):
    """A Q8_0 table of several tiles a CTA: the same hidden rows, the same bits of the logits and the same tokens, and the
    oracle's values."""
    cfg = S.tiny_config(max_ctx=64).replace(lm_format=S.LM_Q8_0, target_dim=target_dim, vocab=40000)
    p = Pair(cfg, 62)
    p.append(0, S.gen_features(S.streams(62)["features"], 30, cfg.feat_dim), 0)
    got, ref = p.draft(0, 123, 30)
    first = p.logits()
    for _ in range(20):
        assert np.array_equal(p.logits(), first)
    for _ in range(50):
        again, _ = p.draft(0, 123, 30, oracle=False)
        assert np.array_equal(again, got)
    assert rel_l2(first, ref.logits) < REL_L2
    assert tokens_match(got, ref.tokens, ref.logits) and np.array_equal(got, np.argmax(first, axis=-1))
    p.close()
