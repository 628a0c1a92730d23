"""The 4-bit cache's refusals that need no device."""
from __future__ import annotations

import ctypes

import pytest

import block_speculative_decoding_fm_gb300 as fm
from block_speculative_decoding_fm_gb300 import build as fmbuild


@pytest.fixture(scope="module")
def lib():
    fmbuild.build()
    return fm.load_library()


@pytest.mark.parametrize("cfg,status", [
    ((1, 1, 1, 96, 64), fm.FM_ERR_UNSUPPORTED), ((0, 1, 1, 64, 64), fm.FM_ERR_INVALID_ARG),
    ((1, 0, 1, 64, 64), fm.FM_ERR_INVALID_ARG), ((1, 1, 0, 64, 64), fm.FM_ERR_INVALID_ARG),
    ((1, 1, 1, 64, 0), fm.FM_ERR_INVALID_ARG), ((1, 1, 1, 64, (1 << 24) + 1), fm.FM_ERR_INVALID_ARG),
    ((1, 65537, 1, 64, 64), fm.FM_ERR_INVALID_ARG), ((1025, 1, 1, 64, 64), fm.FM_ERR_INVALID_ARG)])
def test_create_refuses_before_device_work(lib, cfg, status):
    with pytest.raises(fm.FmError) as e:
        fm.fm_kvq_create(*cfg)
    assert e.value.status == status and lib.fm_kvq_last_error(None)


def test_null_handles(lib):
    bad = fm.FM_ERR_INVALID_ARG
    assert lib.fm_kvq_create(None, None, None) == bad
    out = ctypes.c_void_p(5)
    assert lib.fm_kvq_create(None, None, ctypes.byref(out)) == bad and not out.value
    assert lib.fm_kvq_append(None, 0, 1, None, None, None, None, None, 2, 64, None) == bad
    assert lib.fm_kvq_read(None, 0, 1, None, None, None, None, None, 2, 64, None, 0, None) == bad
    assert lib.fm_kvq_attend(None, 0, 1, None, None, None, 2, 1, 64, 1.0, 0, 0, None, 64, -1.0, None, 0, None) == bad
    assert lib.fm_kvq_set_weights(None, 0, 1, None, None, 0, None) == bad
    assert lib.fm_kvq_evict(None, 0, 1, None, None, 0, 0, None, None) == bad
    n = ctypes.c_int32()
    assert lib.fm_kvq_length(None, 0, 0, ctypes.byref(n)) == bad
    assert lib.fm_kvq_memory_bytes(None, None) == bad
    assert lib.fm_kvq_synchronize(None, None) == bad
    assert lib.fm_kvq_last_error(None) is not None
    lib.fm_kvq_destroy(None)
    fm.fm_kvq_destroy(None)


def test_negative_decay(lib):
    """None leaves the weights alone; a negative number is no decay (the library would leave them alone too)."""
    for d in (-0.5, -1.0, float("-inf")):
        with pytest.raises(fm.FmError) as e:
            fm.fm_mtp_use_kvq(None, None, decay=d)
        assert e.value.status == fm.FM_ERR_INVALID_ARG and "decay" in str(e.value)
