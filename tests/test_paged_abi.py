"""The paged cache's refusals that need no device."""
from __future__ import annotations

import ctypes

import pytest

import block_speculative_decoding_fm_gb300 as fm
from block_speculative_decoding_fm_gb300 import build as fmbuild


@pytest.fixture(scope="module")
def lib():
    fmbuild.build()
    return fm.load_library()


GOOD = dict(n_layers=1, n_pages=4, page_rows=16, n_heads=4, n_kv_heads=2, head_dim=64, dtype=fm.FM_DTYPE_F16, rot_dims=32, rot_layout=0,
            rope_scaling=0, rope_rows=4096, theta=1e4, rope_factor=1.0, rope_low=1.0, rope_high=32.0, rope_gain=1.0, eps=1e-6)
INVALID, UNSUPPORTED = fm.FM_ERR_INVALID_ARG, fm.FM_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


def create(lib, k=1 << 20, v=1 << 21, **change):
    out = ctypes.c_void_p(5)
    g = fm.FmPagedConfig(**(GOOD | change))
    status = lib.fm_paged_create(ctypes.byref(g), k, v, None, ctypes.byref(out))
    assert not out.value
    return status


@pytest.mark.parametrize("change,status", [
    (dict(n_layers=0), INVALID), (dict(n_layers=1025), INVALID), (dict(n_pages=0), INVALID), (dict(page_rows=8), UNSUPPORTED),
    (dict(page_rows=48), UNSUPPORTED), (dict(page_rows=512), UNSUPPORTED), (dict(n_heads=3), INVALID), (dict(n_heads=1), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(n_kv_heads=257, n_heads=257), INVALID), (dict(n_kv_heads=1, n_heads=129), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(dtype=fm.FM_DTYPE_F32), INVALID), (dict(dtype=fm.FM_DTYPE_Q8_0), INVALID),
    (dict(rot_dims=8), INVALID), (dict(rot_dims=-16), INVALID), (dict(rot_dims=80), INVALID), (dict(rot_layout=2), INVALID),
    (dict(rope_scaling=3), INVALID), (dict(theta=0.5), INVALID), (dict(theta=NAN), INVALID), (dict(theta=INF), INVALID),
    (dict(rope_gain=0.0), INVALID), (dict(rope_gain=INF), INVALID), (dict(rope_scaling=1, rope_factor=0.5), INVALID),
    (dict(rope_scaling=2, rope_factor=NAN), INVALID), (dict(rope_scaling=2, rope_rows=0), INVALID),
    (dict(rope_scaling=2, rope_low=32.0), INVALID), (dict(rope_scaling=2, rope_low=-1.0), INVALID),
    (dict(rope_scaling=2, rope_high=INF), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID),
    (dict(n_pages=2 ** 26), UNSUPPORTED), (dict(n_layers=1024, n_pages=2 ** 31 - 1, n_heads=256, n_kv_heads=256), UNSUPPORTED)])
def test_create_refuses_before_device_work(lib, change, status):
    assert create(lib, **change) == status and lib.fm_paged_last_error(None)


@pytest.mark.parametrize("k,v", [(None, 64), (64, None), (64, 64), (72, 128), (64, 136)])
def test_create_refuses_pools(lib, k, v):
    assert create(lib, k, v) == INVALID


def test_null_handles(lib):
    assert lib.fm_paged_create(None, None, None, None, None) == INVALID
    out = ctypes.c_void_p(5)
    assert lib.fm_paged_create(None, None, None, None, ctypes.byref(out)) == INVALID and not out.value
    b, r = fm.FmPagedBatch(), fm.FmPagedRows()
    assert lib.fm_paged_write(None, 0, ctypes.byref(b), None, None, None, 2, None, None, None, None) == INVALID
    assert lib.fm_paged_attend(None, 0, ctypes.byref(b), ctypes.byref(r), ctypes.byref(r), 1.0, 1, 0, 0, None, 0, None) == INVALID
    n = ctypes.c_int64()
    assert lib.fm_paged_workspace_bytes(None, 1, ctypes.byref(n)) == INVALID
    assert lib.fm_paged_get_config(None, None) == INVALID
    assert lib.fm_paged_last_launch_count(None, None) == INVALID
    assert lib.fm_paged_synchronize(None, None) == INVALID
    assert lib.fm_paged_selftest_wait_timeout(None, 1, None) == INVALID
    assert lib.fm_paged_last_error(None) is not None
    lib.fm_paged_destroy(None)
    fm.fm_paged_destroy(None)
