"""The MTP head over a 4-bit cache (fm_mtp_use_kvq) against the oracle.  The rows that the head stores come out of
products whose weights the tensor cores see rounded, so a value next to a border may get the neighbouring code: the
stored rows are compared to within a step of the oracle's, and the oracle then attends over the rows as the cache holds
them, with the head's own bars (h' within 2e-3, tokens exact or excused by the margin)."""
from __future__ import annotations

import numpy as np
import pytest

import fm_synth as S
from gpu_common import REL_L2, rel_l2
from oracle import kvq as Q
from test_gpu_mtp import MtpPair, built, check_tokens, mid_config  # noqa: F401

pytestmark = pytest.mark.gpu


class Held:
    """The oracle's cache array: reads give what the device holds, writes are checked against it."""

    def __init__(self, rows, at):
        self.rows, self.at = rows, at          # [rows][width], and the row of position 0

    def __getitem__(self, i):
        if isinstance(i, tuple):
            return self.rows[self._rows(i[0]), i[1]]
        return self.rows[self._rows(i)]

    def _rows(self, s):
        return slice(s.start + self.at, s.stop + self.at) if isinstance(s, slice) else s + self.at

    def __setitem__(self, i, x):
        held = self[i]
        big = np.abs(x).reshape(-1, Q.GROUP).max(-1)[:, None]
        # half a step of max / 8, one more code for a neighbour, the positive end's 7 / 8, and the product's own error
        assert np.all(np.abs(held - x).reshape(-1, Q.GROUP) <= big / 8 * 1.01 + 2e-3 * big)


class KvqPair(MtpPair):
    def __init__(self, cfg, seed, max_rows, decay=None, layers=2, seqs=2):
        super().__init__(cfg, seed)
        self.c = self.fm.fm_kvq_create(layers, seqs, cfg.n_kv_heads, cfg.head_dim, max_rows)
        self.at = (layers - 1, seqs - 1)
        self.fm.fm_mtp_use_kvq(self.h, self.c, *self.at, decay=decay)

    def held(self, next_pos):
        """The cache as the oracle's state: position p in row p - (next_pos - length)."""
        import torch
        from oracle.mtp import MtpState
        n = self.fm.fm_kvq_length(self.c, *self.at)
        k = torch.zeros((n, self.cfg.n_kv_heads, self.cfg.head_dim), device="cuda")
        v = torch.zeros_like(k)
        self.fm.fm_kvq_read(self.c, self.at[0], [self.at[1]], [0], [n], k, v)
        off = n - next_pos
        return MtpState(*(Held(x.cpu().numpy().astype(np.float64).reshape(n, -1), off) for x in (k, v)))

    def run(self, tokens, pos0, kv_lo=0, oldest=None):
        """A pass on the device, then on the oracle over the rows that the cache now holds (from position `oldest` on)."""
        import torch
        hn = S.gen_mtp_hidden(self.rng, len(tokens), self.cfg.hidden)
        hout = torch.zeros((len(tokens), self.cfg.hidden), dtype=torch.float32, device="cuda")
        drafts = torch.full((len(tokens),), -1, dtype=torch.int32, device="cuda")
        self.fm.fm_mtp_forward(self.h, torch.tensor(tokens, dtype=torch.int32, device="cuda"), torch.from_numpy(hn).cuda(), pos0,
                               kv_lo, hout, drafts)
        self.fm.fm_kvq_synchronize(self.c)
        ref = self.o.forward(self.held(pos0 + len(tokens)), self.o.embed(tokens), hn.astype(np.float64), pos0,
                             kv_lo if oldest is None else oldest)
        assert rel_l2(hout.cpu().numpy(), ref.hout) < REL_L2, rel_l2(hout.cpu().numpy(), ref.hout)
        lg = self.o.logits(ref.hout)
        check_tokens(drafts.cpu().numpy(), np.argmax(lg, axis=-1), lg)


@pytest.mark.parametrize("make", [S.mtp_micro_config, mid_config])
def test_passes(make):
    """Passes of several sizes, a window start, and a rewind (the verify step's), over a cache of more layers and
    sequences; the other ones stay empty."""
    p = KvqPair(make().replace(kv_cap=1), 1301, 80)
    p.run([7, 8, 9, 10], 0)
    for tokens, pos, lo in (([5, 17, 63], 4, 2), ([11], 7, 0), ([12, 13], 6, 1), (list(range(100, 108)), 8, 0)):
        p.run(tokens, pos, lo)
    assert p.fm.fm_kvq_length(p.c, 1, 1) == 16 and p.fm.fm_kvq_length(p.c, 0, 1) == 0
    assert p.fm.fm_mtp_last_launch_count(p.h) > 0
    p.close()


def test_draft_chain():
    """fm_mtp_draft over the 4-bit cache: the chained passes append and attend on the device."""
    import torch
    cfg = S.mtp_micro_config()
    p = KvqPair(cfg, 1302, 64)
    p.run([3, 4, 5, 6], 0)
    hn = S.gen_mtp_hidden(p.rng, 2, cfg.hidden)
    drafts = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    p.fm.fm_mtp_draft(p.h, torch.tensor([21, 22], dtype=torch.int32, device="cuda"), torch.from_numpy(hn).cuda(), 4, 0, 4,
                      drafts)
    p.fm.fm_kvq_synchronize(p.c)
    assert p.fm.fm_kvq_length(p.c, *p.at) == 9
    want, lg, _ = p.o.draft(p.held(9), [21, 22], hn.astype(np.float64), 4, 0, 4)
    check_tokens(drafts.cpu().numpy(), want, lg)
    p.close()


def test_eviction_between_passes():
    """Weights counted in the passes, an eviction in place, and passes at later positions over what is left."""
    import torch
    cfg = S.mtp_micro_config()
    p = KvqPair(cfg, 1303, 200, decay=1.0)
    pos = 0
    for i in range(6):
        p.run([(31 * i + j) % cfg.vocab for j in range(8)], pos)
        pos += 8
    w = torch.zeros((1, cfg.n_kv_heads, 48), device="cuda")
    p.fm.fm_kvq_read(p.c, p.at[0], [p.at[1]], [0], [48], weights=w)
    got = w[0].cpu().numpy()
    assert np.all(got >= 0) and np.allclose(got.sum(-1), 48 * cfg.n_heads / cfg.n_kv_heads, rtol=1e-5)   # each row gives 1 a head
    kept = torch.zeros((1, cfg.n_kv_heads, 20), dtype=torch.int32, device="cuda")
    p.fm.fm_kvq_evict(p.c, p.at[0], [p.at[1]], [p.at[1]], 20, 9, kept)
    for g in range(cfg.n_kv_heads):
        assert np.array_equal(kept[0, g].cpu().numpy(), Q.kept_rows(got[g], 20, 9))
    p.run([1, 2, 3], pos, 0, oldest=pos - 20)             # position p now in row p - 28
    p.run([4, 5], pos + 1, 0, oldest=pos - 20)            # a rewind inside the recent rows
    import block_speculative_decoding_fm_gb300 as fm
    with pytest.raises(fm.FmError) as e:                  # a window start means nothing any more
        p.run([6], pos + 3, 2)
    assert e.value.status == fm.FM_ERR_UNSUPPORTED
    p.close()


def test_full_shape():
    """Heads of 256, 24 over 4, at the sizes of the page's head."""
    p = KvqPair(S.mtp_config(kv_cap=16), 1304, 40, layers=1, seqs=1)
    p.run([1, 2, 3, 4], 0)
    p.run([10, 20], 4)
    p.close()


def test_refusals():
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    cfg = S.mtp_micro_config(kv_cap=16)
    w = S.gen_mtp_weights(cfg, 1305)
    h = fm.fm_mtp_create(cfg, fm.weight_items(w))
    t = torch.zeros((8,), dtype=torch.int32, device="cuda")
    hn = torch.zeros((8, cfg.hidden), dtype=torch.float32, device="cuda")

    def bad(status, f, *a, **k):
        with pytest.raises(fm.FmError) as e:
            f(*a, **k)
        assert e.value.status == status, e.value

    other = fm.fm_kvq_create(1, 1, cfg.n_kv_heads, 128, 20)
    bad(fm.FM_ERR_INVALID_ARG, fm.fm_mtp_use_kvq, h, other)
    c = fm.fm_kvq_create(1, 1, cfg.n_kv_heads, cfg.head_dim, 20)
    bad(fm.FM_ERR_INVALID_ARG, fm.fm_mtp_use_kvq, h, c, 0, 1, next_pos=0)
    bad(fm.FM_ERR_INVALID_ARG, fm.fm_mtp_use_kvq, h, c, 0, 0, decay=float("nan"))
    bad(fm.FM_ERR_INVALID_ARG, fm.fm_mtp_use_kvq, h, c, 0, 0, decay=float("-inf"))
    fm.fm_mtp_forward(h, t[:4], hn[:4], 0, 0)                    # four rows in the head's own cache
    own = fm.fm_mtp_cache(h, 0, 4, np.empty((4, cfg.n_kv_heads * cfg.head_dim), np.float32)).copy()
    fm.fm_mtp_use_kvq(h, c)
    bad(fm.FM_ERR_STATE, fm.fm_mtp_forward, h, t[:1], hn[:1], 1, 0)      # a gap
    fm.fm_mtp_forward(h, t, hn, 0, 0)
    fm.fm_mtp_forward(h, t, hn, 8, 0)
    assert fm.fm_kvq_length(c, 0, 0) == 16
    bad(fm.FM_ERR_CONTEXT_FULL, fm.fm_mtp_forward, h, t[:5], hn[:5], 16, 0)
    d = torch.zeros((8,), dtype=torch.int32, device="cuda")
    bad(fm.FM_ERR_CONTEXT_FULL, fm.fm_mtp_draft, h, t[:2], hn[:2], 16, 0, 4, d)
    assert fm.fm_kvq_length(c, 0, 0) == 16                       # nothing was stored
    bad(fm.FM_ERR_STATE, fm.fm_mtp_cache, h, 0, 4, np.empty((4, cfg.n_kv_heads * cfg.head_dim), np.float32))
    fm.fm_kvq_evict(c, 0, [0], [0], 4, 2)
    bad(fm.FM_ERR_STATE, fm.fm_mtp_forward, h, t[:1], hn[:1], 11, 0)     # past what is left
    fm.fm_mtp_forward(h, t[:1], hn[:1], 16, 0)
    fm.fm_mtp_use_kvq(h, None)                                   # the own cache, as it was
    assert np.array_equal(fm.fm_mtp_cache(h, 0, 4, np.empty_like(own)), own)
    fm.fm_mtp_destroy(h)


def test_sums_past_32_bits():
    """Depths and positions whose sums pass 2^31 are refused before anything is launched, with the 4-bit cache and without."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    cfg = S.mtp_micro_config(kv_cap=16)
    h = fm.fm_mtp_create(cfg, fm.weight_items(S.gen_mtp_weights(cfg, 1306)))
    t = torch.zeros((8,), dtype=torch.int32, device="cuda")
    hn = torch.zeros((8, cfg.hidden), dtype=torch.float32, device="cuda")
    d = torch.zeros((8,), dtype=torch.int32, device="cuda")
    top = 2 ** 31 - 1

    def bad(status, f, *a):
        with pytest.raises(fm.FmError) as e:
            f(*a)
        assert e.value.status == status, e.value
        assert fm.fm_mtp_last_launch_count(h) == 0

    inv = fm.FM_ERR_INVALID_ARG
    bad(inv, fm.fm_mtp_forward, h, t, hn, top, 0)
    bad(inv, fm.fm_mtp_forward, h, t, hn, top - 7, 0)
    for depth in (top, top - 1, top - 8, 0, -1):
        bad(inv, fm.fm_mtp_draft, h, t, hn, 0, 0, depth, d)
        bad(inv, fm.fm_mtp_draft, h, t[:1], hn[:1], 15, 0, depth, d)
    c = fm.fm_kvq_create(1, 1, cfg.n_kv_heads, cfg.head_dim, 40)
    fm.fm_mtp_use_kvq(h, c)
    for depth in (top, top - 1, top - 6, top - 7, 34):
        bad(fm.FM_ERR_CONTEXT_FULL, fm.fm_mtp_draft, h, t, hn, 0, 0, depth, d)
    bad(inv, fm.fm_mtp_draft, h, t, hn, 0, 0, 0, d)
    bad(inv, fm.fm_mtp_draft, h, t, hn, 0, 0, -2 ** 31, d)
    assert fm.fm_kvq_length(c, 0, 0) == 0
    # late positions, as after evictions
    fm.fm_mtp_use_kvq(h, c, next_pos=top - 3)
    bad(inv, fm.fm_mtp_forward, h, t, hn, top - 3, 0)
    bad(inv, fm.fm_mtp_forward, h, t[:4], hn[:4], top - 3, 0)
    bad(inv, fm.fm_mtp_draft, h, t[:2], hn[:2], top - 3, 0, 3, d)
    fm.fm_mtp_forward(h, t[:3], hn[:3], top - 3, 0)
    bad(inv, fm.fm_mtp_forward, h, t[:1], hn[:1], top, 0)
    assert fm.fm_kvq_length(c, 0, 0) == 3
    fm.fm_mtp_destroy(h)


def test_devices():
    """A cache of another device is refused, and so is a pass while another device is the current one."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two devices")
    cfg = S.mtp_micro_config(kv_cap=16)
    h = fm.fm_mtp_create(cfg, fm.weight_items(S.gen_mtp_weights(cfg, 1307)))
    c = fm.fm_kvq_create(1, 1, cfg.n_kv_heads, cfg.head_dim, 20)
    with torch.cuda.device(1):
        other = fm.fm_kvq_create(1, 1, cfg.n_kv_heads, cfg.head_dim, 20)
    with pytest.raises(fm.FmError) as e:
        fm.fm_mtp_use_kvq(h, other)
    assert e.value.status == fm.FM_ERR_INVALID_ARG
    with torch.cuda.device(1), pytest.raises(fm.FmError) as e:        # its rows' buffers would be there
        fm.fm_mtp_use_kvq(h, c)
    assert e.value.status == fm.FM_ERR_INVALID_ARG
    fm.fm_mtp_use_kvq(h, c)
    t = torch.zeros((2,), dtype=torch.int32, device="cuda:0")
    hn = torch.zeros((2, cfg.hidden), dtype=torch.float32, device="cuda:0")
    with torch.cuda.device(1), pytest.raises(fm.FmError) as e:
        fm.fm_mtp_forward(h, t, hn, 0, 0)
    assert e.value.status == fm.FM_ERR_INVALID_ARG and fm.fm_mtp_last_launch_count(h) == 0
    fm.fm_mtp_forward(h, t, hn, 0, 0)
    fm.fm_mtp_destroy(h)


def test_wait_that_gives_up():
    """A bounded wait that gives up: the cache reports it once, and so does the head that uses the cache."""
    import torch
    import block_speculative_decoding_fm_gb300 as fm
    cfg = S.mtp_micro_config(kv_cap=16)
    h = fm.fm_mtp_create(cfg, fm.weight_items(S.gen_mtp_weights(cfg, 1308)))
    c = fm.fm_kvq_create(1, 1, cfg.n_kv_heads, cfg.head_dim, 20)
    none = np.empty((1,), np.float32)

    def timeout(f, *a):
        with pytest.raises(fm.FmError) as e:
            f(*a)
        assert e.value.status == fm.FM_ERR_TIMEOUT, e.value
        f(*a)                                          # reported once

    for budget in (0, 1000001):
        with pytest.raises(fm.FmError) as e:
            fm.fm_kvq_selftest_wait_timeout(c, budget)
        assert e.value.status == fm.FM_ERR_INVALID_ARG
    fm.fm_kvq_synchronize(c)
    fm.fm_kvq_selftest_wait_timeout(c, 20000)
    timeout(fm.fm_kvq_synchronize, c)
    fm.fm_mtp_use_kvq(h, c)
    t = torch.zeros((2,), dtype=torch.int32, device="cuda")
    hn = torch.zeros((2, cfg.hidden), dtype=torch.float32, device="cuda")
    fm.fm_mtp_forward(h, t, hn, 0, 0)
    fm.fm_mtp_cache(h, 0, 0, none)
    fm.fm_kvq_selftest_wait_timeout(c, 20000)
    fm.fm_mtp_forward(h, t, hn, 2, 0)
    timeout(fm.fm_mtp_cache, h, 0, 0, none)
    fm.fm_mtp_forward(h, t, hn, 2, 0)                  # the head and the cache stay usable
    fm.fm_mtp_cache(h, 0, 0, none)
    fm.fm_mtp_destroy(h)
