"""The MTP head over a paged cache: its own head shape, and calls that fail."""
from __future__ import annotations

import ctypes

import pytest

import fm_synth as S
from gpu_common import REL_L2, rel_l2
from test_gpu_kvq_calls import runtime
from test_gpu_mtp import MtpPair, built  # noqa: F401
from test_gpu_mtp_paged import PagedPair

pytestmark = pytest.mark.gpu


def wide_config():
    """24 query heads over 4 of 256, 64 rotated dims: the full head's attention over a narrower stream."""
    return S.MtpConfig(hidden=1024, inter=2048, n_heads=24, n_kv_heads=4, head_dim=256, rot_dims=64, theta=1e7, vocab=8192, kv_cap=160)


def test_full_heads():
    """Single rows (the few-rows kernel) and eight (tiles of 128 rows), pages in any order."""
    p = PagedPair(wide_config(), 1411, pages=10)
    pos = 0
    for n in (8, 1, 8, 8, 3, 1, 8, 8, 8, 2, 1, 8, 8):
        p.run([100 + pos + i for i in range(n)], pos)
        pos += n
    p.close()


def test_full_heads_window():
    p = PagedPair(wide_config(), 1412, window=7)
    for pos in range(20):
        p.run([20 + pos], pos, max(0, pos - 6))
    p.close()


def test_a_failed_call_changes_nothing():
    """fm_mtp_use_paged whose allocations fail (they are refused while the thread captures): the head goes on over what it had,
    and takes the cache when it is asked again."""
    import torch
    cfg = S.mtp_micro_config()
    p = MtpPair(cfg, 1413)
    p.forward([1, 2, 3], 0, 0)
    k, v = (torch.zeros((1, 4, cfg.n_kv_heads, 16, cfg.head_dim), dtype=torch.float16, device="cuda") for _ in "kv")
    c = p.fm.fm_paged_create(k, v, cfg.n_heads, rot_dims=cfg.rot_dims, layout=p.fm.FM_ROPE_HALF, theta=cfg.theta, eps=cfg.eps)
    table = torch.arange(4, dtype=torch.int32, device="cuda")
    lib, stream, graph = runtime(), torch.cuda.Stream(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert lib.cudaStreamBeginCapture(ctypes.c_void_p(stream.cuda_stream), 1) == 0      # (this thread's calls alone)
    try:
        with pytest.raises(p.fm.FmError) as e:
            p.fm.fm_mtp_use_paged(p.h, c, 0, table)
    finally:
        lib.cudaStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph))
        if graph.value:
            lib.cudaGraphDestroy(graph)
        lib.cudaGetLastError()
    assert e.value.status == p.fm.FM_ERR_OOM
    out, _, ref = p.forward([4], 3, 0)
    assert rel_l2(out, ref.hout) < REL_L2 and not k.any()
    p.fm.fm_mtp_use_paged(p.h, c, 0, table)
    t, hn = torch.tensor([9], dtype=torch.int32, device="cuda"), torch.from_numpy(S.gen_mtp_hidden(p.rng, 1, cfg.hidden)).cuda()
    p.fm.fm_mtp_forward(p.h, t, hn, 0, 0)
    p.fm.fm_paged_synchronize(c)
    assert k[0, 0, :, 0].any()
    with pytest.raises(p.fm.FmError):
        p.fm.fm_mtp_use_paged(p.h, c, 1, table)
    before = k.clone()
    p.fm.fm_mtp_forward(p.h, t, hn, 1, 0)
    p.fm.fm_paged_synchronize(c)
    assert k[0, 0, :, 1].any() and torch.equal(k[0, 0, :, 0], before[0, 0, :, 0])
    p.close()


def test_beside_other_launches_with_tensor_memory():
    """Chunks of head dim 64, whose CTAs leave room on an SM, and passes of a head, one behind the other in a stream: each gets its
    tensor memory, and what it gives alone."""
    import torch
    from paged_common import Batch
    cfg = S.mtp_micro_config()
    p = MtpPair(cfg, 1414)
    B = Batch([(40, 300), (3, 900), (64, 10)], 2, 2, 64, 32, torch.bfloat16, seed=59).create().fill_rows()
    q = B.queries()
    t, hn = torch.tensor([9, 8, 7], dtype=torch.int32, device="cuda"), torch.from_numpy(S.gen_mtp_hidden(p.rng, 3, cfg.hidden)).cuda()
    results = []
    for _ in range(60):
        out, h = torch.zeros_like(q), torch.zeros((3, cfg.hidden), device="cuda")
        p.fm.fm_paged_attend(B.c, 0, B.b, q, out)
        p.fm.fm_mtp_forward(p.h, t, hn, 0, 0, h)
        p.fm.fm_paged_attend(B.c, 0, B.b, q, out)
        results.append((out, h))
    p.fm.fm_paged_synchronize(B.c)
    for out, h in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(h, results[0][1])
    alone = torch.zeros_like(q)
    p.fm.fm_paged_attend(B.c, 0, B.b, q, alone)
    torch.cuda.synchronize()
    assert torch.equal(alone, results[0][0])
    p.close()
