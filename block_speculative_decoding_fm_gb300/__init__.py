"""Python binding of libfm.so (include/fm.h): argument marshalling only.

Every function below has the name of the C entry point it calls and does
nothing but convert arguments (numpy / torch tensors, streams) and turn a
non-zero status into an ``FmError``.  All compute runs in the library's CUDA
kernels; there is no CPU fallback: if the library is missing or cannot load,
``load_library`` raises.  PyTorch supplies device memory and streams.
"""
from __future__ import annotations

import array
import ctypes
import os
from typing import Dict, Iterable, Optional, Sequence, Tuple

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfm.so")

# status codes (fm_status)
FM_OK, FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED, FM_ERR_OOM, FM_ERR_CONTEXT_FULL, FM_ERR_STATE, FM_ERR_CUDA, \
    FM_ERR_TIMEOUT = range(8)
FM_VARIANT_FLASHMAP, FM_VARIANT_DFLASH = 0, 1
FM_LM_BF16, FM_LM_Q8_0 = 0, 1
FM_DTYPE_BF16, FM_DTYPE_Q8_0, FM_DTYPE_F32, FM_DTYPE_F16 = 0, 1, 2, 3
FM_DEBUG_HIDDEN, FM_DEBUG_HEAD_OUT, FM_DEBUG_LOGITS, FM_DEBUG_CACHE_K, FM_DEBUG_CACHE_V, FM_DEBUG_H0, \
    FM_DEBUG_STEP_TRACE = range(7)
FM_DEBUG_KEEP_HIDDEN = 1
FM_DEBUG_PROFILE = 2
FM_DEBUG_TRACE = 4

EXPORTS = ["fm_create", "fm_time_conditioning", "fm_context_append", "fm_context_append_batched", "fm_draft",
           "fm_context_append_host", "fm_context_append_batched_host", "fm_draft_host", "fm_draft_pruned",
           "fm_accept", "fm_accept_batched", "fm_lm_head_argmax_noalloc", "fm_synchronize",
           "fm_selftest_wait_timeout", "fm_debug_copy", "fm_set_debug", "fm_get_length", "fm_memory_bytes",
           "fm_last_launch_count", "fm_profile_read", "fm_status_str", "fm_last_error", "fm_destroy",
           "fm_policy_init", "fm_policy_next", "fm_policy_after_round", "fm_policy_after_plain",
           "fm_mtp_create", "fm_mtp_forward", "fm_mtp_draft", "fm_mtp_cache", "fm_mtp_last_launch_count",
           "fm_mtp_last_error", "fm_mtp_destroy",
           "fm_kvq_create", "fm_kvq_append", "fm_kvq_read", "fm_kvq_attend", "fm_kvq_set_weights", "fm_kvq_evict",
           "fm_kvq_length", "fm_kvq_get_config", "fm_kvq_last_launch_count", "fm_mtp_use_kvq",
           "fm_kvq_memory_bytes", "fm_kvq_synchronize", "fm_kvq_selftest_wait_timeout", "fm_kvq_last_error", "fm_kvq_destroy",
           "fm_paged_create", "fm_paged_write", "fm_paged_attend", "fm_paged_workspace_bytes", "fm_paged_get_config",
           "fm_paged_last_launch_count", "fm_paged_synchronize", "fm_paged_selftest_wait_timeout", "fm_paged_last_error",
           "fm_paged_destroy", "fm_mtp_use_paged"]
FM_ROPE_INTERLEAVED, FM_ROPE_HALF = 0, 1
FM_ROPE_PLAIN, FM_ROPE_LINEAR, FM_ROPE_BY_PARTS = 0, 1, 2


class FmConfig(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("dim", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_layers", ctypes.c_int32), ("ff_dim", ctypes.c_int32),
                ("block", ctypes.c_int32), ("target_dim", ctypes.c_int32), ("n_taps", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("lm_format", ctypes.c_int32), ("max_ctx", ctypes.c_int32),
                ("max_seqs", ctypes.c_int32), ("rope_theta", ctypes.c_float), ("ln_eps", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("qk_eps", ctypes.c_float)]


class FmTensor(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("data", ctypes.c_void_p), ("nbytes", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("on_device", ctypes.c_int32)]


class FmKernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int32), ("ms", ctypes.c_float),
                ("bytes", ctypes.c_double)]


class FmVerifyPolicy(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int32), ("verify", ctypes.c_int32), ("fallback", ctypes.c_int32),
                ("probe_every", ctypes.c_int32), ("ema", ctypes.c_double), ("ema_tokens", ctypes.c_double),
                ("round_ms", ctypes.c_double), ("step_ms", ctypes.c_double), ("plain_left", ctypes.c_int32),
                ("rounds", ctypes.c_int32), ("catch_up", ctypes.c_int32), ("pad", ctypes.c_int32)]


FM_ACT_ROUND, FM_ACT_PLAIN, FM_ACT_PLAIN_LIMIT = 0, 1, 2


class FmMtpConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rot_dims", ctypes.c_int32),
                ("theta", ctypes.c_float), ("eps", ctypes.c_float), ("vocab", ctypes.c_int32),
                ("kv_cap", ctypes.c_int32), ("max_rows", ctypes.c_int32)]


class FmKvqConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_seqs", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("max_rows", ctypes.c_int32)]


class FmPagedConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_rows", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("rot_dims", ctypes.c_int32), ("rot_layout", ctypes.c_int32),
                ("rope_scaling", ctypes.c_int32), ("rope_rows", ctypes.c_int32), ("theta", ctypes.c_float),
                ("rope_factor", ctypes.c_float), ("rope_low", ctypes.c_float), ("rope_high", ctypes.c_float),
                ("rope_gain", ctypes.c_float), ("eps", ctypes.c_float)]


class FmPagedBatch(ctypes.Structure):
    _fields_ = [("starts", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_ld", ctypes.c_int64), ("n_seqs", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
                ("table_pages", ctypes.c_int32), ("max_new", ctypes.c_int32)]


class FmPagedRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class FmError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfm.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run block_speculative_decoding_fm_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "fm_create": (I32, [ctypes.POINTER(FmConfig), ctypes.POINTER(FmTensor), I32, P, P, ctypes.POINTER(P)]),
        "fm_time_conditioning": (I32, [ctypes.POINTER(FmConfig), ctypes.POINTER(FmTensor), I32, I32, I32,
                                       ctypes.c_float, ctypes.c_float, ctypes.c_float, P, P]),
        "fm_context_append": (I32, [P, I32, P, I32, I32, P]),
        "fm_context_append_batched": (I32, [P, I32, P, P, P, P, P]),
        "fm_draft": (I32, [P, I32, P, P, P, P, P]),
        "fm_context_append_host": (I32, [P, I32, P, I32, I32, P]),
        "fm_context_append_batched_host": (I32, [P, I32, P, P, P, P, P]),
        "fm_draft_host": (I32, [P, I32, P, P, P, P, P]),
        "fm_draft_pruned": (I32, [P, I32, I32, I32, P, ctypes.c_float, P, P, P, P]),
        "fm_accept": (I32, [P, P, I32, P, P]),
        "fm_accept_batched": (I32, [P, I32, P, P, P, P, P, P]),
        "fm_lm_head_argmax_noalloc": (I32, [P, P, I32, P, P]),
        "fm_synchronize": (I32, [P, P]),
        "fm_selftest_wait_timeout": (I32, [P, I32, P]),
        "fm_debug_copy": (I32, [P, I32, I32, I32, I64, P, I64, P]),
        "fm_set_debug": (I32, [P, I32]),
        "fm_get_length": (I32, [P, I32, ctypes.POINTER(I32)]),
        "fm_memory_bytes": (I32, [P, ctypes.POINTER(I64)]),
        "fm_last_launch_count": (I32, [P, ctypes.POINTER(I32)]),
        "fm_profile_read": (I32, [P, ctypes.POINTER(FmKernelTime), I32, ctypes.POINTER(I32)]),
        "fm_status_str": (ctypes.c_char_p, [I32]),
        "fm_last_error": (ctypes.c_char_p, [P]),
        "fm_destroy": (None, [P]),
        "fm_policy_init": (I32, [ctypes.POINTER(FmVerifyPolicy), I32, I32, I32, I32]),
        "fm_policy_next": (I32, [ctypes.POINTER(FmVerifyPolicy), I32, I32, ctypes.POINTER(I32), ctypes.POINTER(I32)]),
        "fm_policy_after_round": (I32, [ctypes.POINTER(FmVerifyPolicy), I32, ctypes.c_double]),
        "fm_policy_after_plain": (I32, [ctypes.POINTER(FmVerifyPolicy), ctypes.c_double, I32]),
        "fm_mtp_create": (I32, [ctypes.POINTER(FmMtpConfig), ctypes.POINTER(FmTensor), I32, P, ctypes.POINTER(P)]),
        "fm_mtp_forward": (I32, [P, I32, P, P, I32, I32, P, P, P]),
        "fm_mtp_draft": (I32, [P, I32, P, P, I32, I32, I32, P, P]),
        "fm_mtp_cache": (I32, [P, I32, I32, P, P]),
        "fm_mtp_last_launch_count": (I32, [P, ctypes.POINTER(I32)]),
        "fm_mtp_last_error": (ctypes.c_char_p, [P]),
        "fm_mtp_destroy": (None, [P]),
        "fm_kvq_create": (I32, [ctypes.POINTER(FmKvqConfig), P, ctypes.POINTER(P)]),
        "fm_kvq_append": (I32, [P, I32, I32, P, P, P, P, P, I32, I64, P]),
        "fm_kvq_read": (I32, [P, I32, I32, P, P, P, P, P, I32, I64, P, I64, P]),
        "fm_kvq_attend": (I32, [P, I32, I32, P, P, P, I32, I32, I64, ctypes.c_float, I32, I32, P, I64, ctypes.c_float,
                                P, I64, P]),
        "fm_kvq_set_weights": (I32, [P, I32, I32, P, P, I64, P]),
        "fm_kvq_evict": (I32, [P, I32, I32, P, P, I32, I32, P, P]),
        "fm_kvq_length": (I32, [P, I32, I32, ctypes.POINTER(I32)]),
        "fm_kvq_get_config": (I32, [P, ctypes.POINTER(FmKvqConfig)]),
        "fm_kvq_last_launch_count": (I32, [P, ctypes.POINTER(I32)]),
        "fm_mtp_use_kvq": (I32, [P, P, I32, I32, I64, ctypes.c_float]),
        "fm_kvq_memory_bytes": (I32, [P, ctypes.POINTER(I64)]),
        "fm_kvq_synchronize": (I32, [P, P]),
        "fm_kvq_selftest_wait_timeout": (I32, [P, I32, P]),
        "fm_kvq_last_error": (ctypes.c_char_p, [P]),
        "fm_kvq_destroy": (None, [P]),
        "fm_paged_create": (I32, [ctypes.POINTER(FmPagedConfig), P, P, P, ctypes.POINTER(P)]),
        "fm_paged_write": (I32, [P, I32, P, P, P, P, I32, P, P, P, P]),
        "fm_paged_attend": (I32, [P, I32, P, P, P, ctypes.c_float, I32, I32, I32, P, I64, P]),
        "fm_paged_workspace_bytes": (I32, [P, I32, ctypes.POINTER(I64)]),
        "fm_paged_get_config": (I32, [P, ctypes.POINTER(FmPagedConfig)]),
        "fm_paged_last_launch_count": (I32, [P, ctypes.POINTER(I32)]),
        "fm_paged_synchronize": (I32, [P, P]),
        "fm_paged_selftest_wait_timeout": (I32, [P, I32, P]),
        "fm_paged_last_error": (ctypes.c_char_p, [P]),
        "fm_paged_destroy": (None, [P]),
        "fm_mtp_use_paged": (I32, [P, P, I32, P, I32, I32, I32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


_raw_stream = None   # torch's current stream as an integer; None: not looked up yet, or no CUDA


def _find_raw_stream():
    """The quickest way this torch has to the current stream's handle (a tenth of a stream object's cost), or None
    without CUDA."""
    global _raw_stream
    import torch
    if torch.cuda.is_available():
        get, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if get is not None and device is not None:
            torch.cuda.current_stream()   # (sets CUDA up)
            _raw_stream = lambda: get(device())
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream
    return _raw_stream


def _stream(stream) -> Optional[int]:
    if stream is None:
        raw = _raw_stream or _find_raw_stream()
        return raw() if raw is not None else None
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, handle=None):
    if status != FM_OK:
        lib = load_library()
        msg = lib.fm_last_error(handle).decode() if handle is not None else lib.fm_last_error(None).decode()
        raise FmError(status, f"{lib.fm_status_str(status).decode()}: {msg}")


def make_config(cfg) -> FmConfig:
    """An FmConfig from any object with the fm_config fields."""
    return FmConfig(cfg.variant, cfg.dim, cfg.n_heads, cfg.head_dim, cfg.n_layers, cfg.ff_dim, cfg.block,
                    cfg.target_dim, cfg.n_taps, cfg.vocab, cfg.lm_format, cfg.max_ctx, cfg.max_seqs,
                    cfg.rope_theta, cfg.ln_eps, cfg.rms_eps, cfg.qk_eps)


def _tensor_array(weights):
    items = list(weights)
    keep = []
    arr = (FmTensor * max(1, len(items)))()
    for i, (name, data, dtype) in enumerate(items):
        on_dev = 0
        if isinstance(data, np.ndarray):
            data = np.ascontiguousarray(data)
            nbytes = data.nbytes
        else:
            on_dev = 1 if data.is_cuda else 0
            nbytes = data.numel() * data.element_size()
        keep.append(data)
        bname = name.encode()
        keep.append(bname)
        arr[i] = FmTensor(bname, _ptr(data), nbytes, dtype, on_dev)
    return arr, len(items), keep


def fm_time_conditioning(cfg, weights: Iterable[Tuple[str, object, int]], time_dim: int, cond_dim: int,
                         time_scale: float, s: float, t: float, table, stream=None) -> None:
    """The adaLN table of the jump s -> t into ``table`` (a CUDA float32
    tensor of (3 n_layers + 1) * 3 * dim values)."""
    lib = load_library()
    arr, n, keep = _tensor_array(weights)
    c = make_config(cfg)
    _check(lib.fm_time_conditioning(ctypes.byref(c), arr, n, time_dim, cond_dim, time_scale, s, t, _ptr(table),
                                    _stream(stream)))


def fm_create(cfg, weights: Iterable[Tuple[str, object, int]], modulation=None, stream=None) -> ctypes.c_void_p:
    """weights: (name, array, FM_DTYPE_*) triples; arrays are host numpy
    arrays or CUDA tensors (their raw bytes are passed).  modulation: a host
    array or a CUDA float32 tensor."""
    lib = load_library()
    arr, n_items, keep = _tensor_array(weights)
    items = range(n_items)
    mod = None
    if modulation is not None:
        mod = modulation if hasattr(modulation, "data_ptr") else np.ascontiguousarray(modulation, dtype=np.float32)
        keep.append(mod)
    c = make_config(cfg)
    h = ctypes.c_void_p()
    _check(lib.fm_create(ctypes.byref(c), arr, len(items), _ptr(mod), _stream(stream), ctypes.byref(h)))
    h._fm_target_dim = int(cfg.target_dim)
    h._fm_block = int(cfg.block)
    h._fm_feat = int(cfg.n_taps) * int(cfg.target_dim)
    return h


def fm_context_append(h, seq: int, feats, n_rows: int, start_pos: int, stream=None) -> None:
    lib = load_library()
    _check(lib.fm_context_append(h, seq, _ptr(feats), n_rows, start_pos, _stream(stream)), h)


def fm_context_append_batched(h, seq_ids: Sequence[int], feats, n_rows: Sequence[int], starts: Sequence[int],
                              stream=None) -> None:
    lib = load_library()
    n = len(seq_ids)
    ids = np.ascontiguousarray(seq_ids, np.int32)
    nr = np.ascontiguousarray(n_rows, np.int32)
    st = np.ascontiguousarray(starts, np.int32)
    _check(lib.fm_context_append_batched(h, n, _ptr(ids), _ptr(feats), _ptr(nr), _ptr(st), _stream(stream)), h)


def fm_draft(h, seq_ids: Sequence[int], anchors: Sequence[int], pos: Sequence[int], tokens, stream=None) -> None:
    """tokens: a CUDA int32 tensor [n_seqs, block] that receives the drafts."""
    lib = load_library()
    ids = np.ascontiguousarray(seq_ids, np.int32)
    an = np.ascontiguousarray(anchors, np.int32)
    ps = np.ascontiguousarray(pos, np.int32)
    _check(lib.fm_draft(h, len(ids), _ptr(ids), _ptr(an), _ptr(ps), _ptr(tokens), _stream(stream)), h)


def _host_buffer(x, dtype, what: str, need: int):
    """A host buffer for the host-buffer calls: a C-contiguous numpy array or
    CPU tensor of dtype with at least need elements (pinned memory keeps the
    copy asynchronous)."""
    if isinstance(x, np.ndarray):
        ok, size = x.dtype == dtype and x.flags["C_CONTIGUOUS"], x.size
    else:
        ok = not getattr(x, "is_cuda", True) and x.is_contiguous() and str(x.dtype) == "torch." + np.dtype(dtype).name
        size = x.numel() if ok else 0
    if not ok:
        raise ValueError(f"{what} must be a contiguous {np.dtype(dtype).name} host array or CPU tensor")
    if size < need:
        raise ValueError(f"{what} holds {size} values, fewer than the call's {need}")
    return x


def fm_context_append_host(h, seq: int, feats, n_rows: int, start_pos: int, stream=None) -> None:
    """fm_context_append with the rows in host memory (copied on the stream)."""
    lib = load_library()
    f = None if n_rows <= 0 else _host_buffer(feats, np.float32, "feature rows", n_rows * h._fm_feat)
    _check(lib.fm_context_append_host(h, seq, _ptr(f), n_rows, start_pos, _stream(stream)), h)


def fm_context_append_batched_host(h, seq_ids: Sequence[int], feats, n_rows: Sequence[int], starts: Sequence[int],
                                   stream=None) -> None:
    lib = load_library()
    ids = np.ascontiguousarray(seq_ids, np.int32)
    nr = np.ascontiguousarray(n_rows, np.int32)
    st = np.ascontiguousarray(starts, np.int32)
    total = int(np.maximum(nr, 0).sum())
    f = None if total == 0 else _host_buffer(feats, np.float32, "feature rows", total * h._fm_feat)
    _check(lib.fm_context_append_batched_host(h, len(ids), _ptr(ids), _ptr(f), _ptr(nr), _ptr(st),
                                              _stream(stream)), h)


def fm_draft_host(h, seq_ids: Sequence[int], anchors: Sequence[int], pos: Sequence[int], tokens, stream=None) -> None:
    """tokens: host int32 [n_seqs, block] (numpy array or CPU tensor, pinned for an
    asynchronous copy); complete once the stream has passed the call."""
    lib = load_library()
    ids = np.ascontiguousarray(seq_ids, np.int32)
    an = np.ascontiguousarray(anchors, np.int32)
    ps = np.ascontiguousarray(pos, np.int32)
    _host_buffer(tokens, np.int32, "tokens", len(ids) * h._fm_block)
    _check(lib.fm_draft_host(h, len(ids), _ptr(ids), _ptr(an), _ptr(ps), _ptr(tokens), _stream(stream)), h)


def fm_draft_pruned(h, seq: int, anchor: int, pos: int, tokens, conf=None, length=None, thresholds=None,
                    min_conf: Optional[float] = None, stream=None) -> None:
    """The DFlash draft through the sequential head with confidence pruning.
    tokens: a CUDA int32 tensor [block]; conf: a CUDA float32 tensor [block] or
    None; length: a CUDA int32 tensor [1] or None.  thresholds: per-position
    thresholds (a sequence of block floats, NaN for none) or None, in which
    case min_conf (None: no pruning) applies to every position."""
    lib = load_library()
    thr = None if thresholds is None else np.ascontiguousarray(thresholds, np.float32)
    mc = float("nan") if min_conf is None else float(min_conf)
    _check(lib.fm_draft_pruned(h, seq, anchor, pos, _ptr(thr), mc, _ptr(tokens), _ptr(conf), _ptr(length),
                               _stream(stream)), h)


def fm_accept(draft: Sequence[int], target: Sequence[int], k: int) -> Tuple[int, int]:
    lib = load_library()
    d = np.ascontiguousarray(draft, np.int32)
    t = np.ascontiguousarray(target, np.int32)
    acc, bonus = ctypes.c_int32(), ctypes.c_int32()
    _check(lib.fm_accept(_ptr(d), _ptr(t), k, ctypes.byref(acc), ctypes.byref(bonus)))
    return acc.value, bonus.value


def fm_accept_batched(h, draft, target, k, n_accepted, bonus, stream=None) -> None:
    lib = load_library()
    _check(lib.fm_accept_batched(h, draft.shape[0], _ptr(draft), _ptr(target), _ptr(k), _ptr(n_accepted),
                                 _ptr(bonus), _stream(stream)), h)


def fm_lm_head_argmax_noalloc(h, y, tokens, stream=None) -> None:
    """The fused lm_head + argmax on caller rows, for callers that must not
    allocate device memory while they run (the library keeps its scratch in
    static device memory).  y: a CUDA float32 tensor [n_rows, target_dim]
    (n_rows <= 16); tokens: a CUDA int32 tensor [n_rows] that receives the
    argmax over the token table.  The first call on a device does a one-time
    set-up, so make it before any stream capture; overlapping calls race."""
    import torch
    if not (isinstance(y, torch.Tensor) and isinstance(tokens, torch.Tensor)):
        raise ValueError("y and tokens must be torch tensors")
    if not (y.is_cuda and tokens.is_cuda):
        raise ValueError("y and tokens must be CUDA tensors")
    if y.dtype != torch.float32 or tokens.dtype != torch.int32:
        raise ValueError("y must be float32 and tokens int32")
    if y.dim() != 2 or not y.is_contiguous() or not tokens.is_contiguous():
        raise ValueError("y must be a contiguous [n_rows, target_dim] tensor and tokens contiguous")
    width = getattr(h, "_fm_target_dim", None)
    if width is not None and y.shape[1] != width:
        raise ValueError(f"y has {y.shape[1]} columns, the drafter's target_dim is {width}")
    if tokens.numel() < y.shape[0]:
        raise ValueError("tokens holds fewer entries than y has rows")
    _check(load_library().fm_lm_head_argmax_noalloc(h, _ptr(y), y.shape[0], _ptr(tokens), _stream(stream)), h)


def fm_synchronize(h, stream=None) -> None:
    """Wait for the stream; raise FmError(FM_ERR_TIMEOUT) if a device-side
    bounded wait gave up since the last check."""
    _check(load_library().fm_synchronize(h, _stream(stream)), h)


def fm_selftest_wait_timeout(h, budget_us: int, stream=None) -> None:
    """Launch a wait that cannot complete, bounded by budget_us (the failure
    path of the bounded waits); the next fm_synchronize reports it."""
    _check(load_library().fm_selftest_wait_timeout(h, budget_us, _stream(stream)), h)


def fm_debug_copy(h, what: int, seq: int, index: int, out: np.ndarray, offset: int = 0, stream=None) -> np.ndarray:
    lib = load_library()
    _check(lib.fm_debug_copy(h, what, seq, index, offset, _ptr(out), out.nbytes, _stream(stream)), h)
    return out


def fm_set_debug(h, flags: int) -> None:
    _check(load_library().fm_set_debug(h, flags), h)


def fm_get_length(h, seq: int) -> int:
    v = ctypes.c_int32()
    _check(load_library().fm_get_length(h, seq, ctypes.byref(v)), h)
    return v.value


def fm_memory_bytes(h) -> int:
    v = ctypes.c_int64()
    _check(load_library().fm_memory_bytes(h, ctypes.byref(v)), h)
    return v.value


def fm_last_launch_count(h) -> int:
    v = ctypes.c_int32()
    _check(load_library().fm_last_launch_count(h, ctypes.byref(v)), h)
    return v.value


def fm_profile_read(h):
    """{kernel name: (launches, total ms, total algorithmic bytes)} since the last read."""
    lib = load_library()
    buf = (FmKernelTime * 64)()
    n = ctypes.c_int32()
    _check(lib.fm_profile_read(h, buf, 64, ctypes.byref(n)), h)
    return {buf[i].name.decode(): (buf[i].launches, buf[i].ms, buf[i].bytes) for i in range(min(n.value, 64))}


def fm_destroy(h) -> None:
    if h is not None:
        load_library().fm_destroy(h)


def weight_items(tensors: Dict[str, object]):
    """(name, array, dtype) triples from name -> object with .data / .dtype."""
    return [(n, t.data, t.dtype) for n, t in tensors.items()]


def _mtp_check(status: int, m=None):
    if status != FM_OK:
        lib = load_library()
        raise FmError(status, f"{lib.fm_status_str(status).decode()}: {lib.fm_mtp_last_error(m).decode()}")


def fm_mtp_create(cfg, weights: Iterable[Tuple[str, object, int]], stream=None) -> ctypes.c_void_p:
    """The MTP draft head.  cfg: any object with the fm_mtp_config fields;
    weights: (name, array, FM_DTYPE_*) triples (host arrays or CUDA tensors)."""
    lib = load_library()
    arr, n_items, keep = _tensor_array(weights)
    c = FmMtpConfig(cfg.hidden, cfg.inter, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.rot_dims, cfg.theta, cfg.eps,
                    cfg.vocab, cfg.kv_cap, cfg.max_rows)
    m = ctypes.c_void_p()
    _mtp_check(lib.fm_mtp_create(ctypes.byref(c), arr, n_items, _stream(stream), ctypes.byref(m)))
    return m


def fm_mtp_forward(m, tokens, hn, pos0: int, kv_lo: int, hout=None, drafts=None, stream=None) -> None:
    """One pass over len(tokens) rows.  tokens: CUDA int32 [M]; hn: CUDA float32
    [M, H]; hout: CUDA float32 [M, H] or None; drafts: CUDA int32 [M] or None."""
    _mtp_check(load_library().fm_mtp_forward(m, int(tokens.shape[0]), _ptr(tokens), _ptr(hn), pos0, kv_lo, _ptr(hout),
                                             _ptr(drafts), _stream(stream)), m)


def fm_mtp_draft(m, tokens, hn, pos0: int, kv_lo: int, depth: int, drafts, stream=None) -> None:
    """A pass over the pending rows then depth - 1 chained single-row passes;
    drafts: CUDA int32 [depth]."""
    _mtp_check(load_library().fm_mtp_draft(m, int(tokens.shape[0]), _ptr(tokens), _ptr(hn), pos0, kv_lo, depth,
                                           _ptr(drafts), _stream(stream)), m)


def fm_mtp_cache(m, which: int, rows: int, out: np.ndarray, stream=None) -> np.ndarray:
    """Copy K (0) or V (1) cache rows [0, rows) into a host float32 array."""
    _mtp_check(load_library().fm_mtp_cache(m, which, rows, _ptr(out), _stream(stream)), m)
    return out


def fm_mtp_last_launch_count(m) -> int:
    n = ctypes.c_int32()
    _mtp_check(load_library().fm_mtp_last_launch_count(m, ctypes.byref(n)), m)
    return n.value


def fm_mtp_destroy(m) -> None:
    if m is not None:
        load_library().fm_mtp_destroy(m)


def fm_policy_init(block: int, verify: int = 0, fallback: bool = True, probe_every: int = 16) -> FmVerifyPolicy:
    p = FmVerifyPolicy()
    _check(load_library().fm_policy_init(ctypes.byref(p), block, verify, 1 if fallback else 0, probe_every))
    return p


def fm_policy_next(p: FmVerifyPolicy, position: int, max_ctx: int) -> Tuple[int, int]:
    """(action, k): FM_ACT_ROUND with the verify length, or a plain step."""
    a, k = ctypes.c_int32(), ctypes.c_int32()
    _check(load_library().fm_policy_next(ctypes.byref(p), position, max_ctx, ctypes.byref(a), ctypes.byref(k)))
    return a.value, k.value


def fm_policy_after_round(p: FmVerifyPolicy, accepted: int, ms: float) -> None:
    _check(load_library().fm_policy_after_round(ctypes.byref(p), accepted, ms))


def fm_policy_after_plain(p: FmVerifyPolicy, ms: float, rows_handed: bool) -> None:
    _check(load_library().fm_policy_after_plain(ctypes.byref(p), ms, 1 if rows_handed else 0))


class KvqCache(ctypes.c_void_p):
    """The handle of a 4-bit KV cache; freed by fm_kvq_destroy, or with the last reference to it."""

    def __del__(self):
        if self.value and _lib is not None:
            _lib.fm_kvq_destroy(self)
            self.value = None


def _kvq_check(status: int, c=None):
    if status != FM_OK:
        lib = load_library()
        raise FmError(status, f"{lib.fm_status_str(status).decode()}: {lib.fm_kvq_last_error(c).decode()}")


def _ints(x, n: int, what: str):
    """A host int32 array of n values for the library."""
    if len(x) != n:
        raise ValueError(f"{what}: {len(x)} values for {n} sequences")
    return array.array("i", x)   # (a fifth of the time that a ctypes array takes)


def _addr(x: array.array) -> int:
    """Where x's values are; the caller keeps x."""
    return x.buffer_info()[0]


_kvq_types = {}   # torch dtype -> FM_DTYPE_*


def _kvq_rows(x, rows: int, heads: Optional[int], c, what: str):
    """(pointer, dtype, heads, row stride) of a tensor [>= rows, heads, head_dim] on the cache's device whose rows are
    whole: the last two axes contiguous, any stride between rows."""
    head_dim = c._head_dim
    if not _kvq_types:
        import torch
        _kvq_types.update({torch.float32: FM_DTYPE_F32, torch.float16: FM_DTYPE_F16, torch.bfloat16: FM_DTYPE_BF16})
    dtype = _kvq_types.get(x.dtype)
    if dtype is None or x.get_device() != c._device:
        raise ValueError(f"{what} must be a float32, float16 or bfloat16 tensor on cuda:{c._device}")
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[2] != head_dim or (heads is not None and shape[1] != heads) or shape[0] < rows:
        raise ValueError(f"{what} has shape {tuple(shape)}, expected [{rows}, {heads or 'heads'}, {head_dim}]")
    if rows and (stride[2] != 1 or (shape[1] > 1 and stride[1] != head_dim)):
        raise ValueError(f"{what}: a row's heads must be contiguous")
    return x.data_ptr(), dtype, shape[1], stride[0] if shape[0] > 1 else shape[1] * head_dim


def _kvq_weights(x, n: int, c, what: str):
    """(pointer, row stride) of a contiguous float32 tensor [n, n_kv_heads, rows] on the cache's device, or of None."""
    if x is None:
        return None, 0
    import torch
    if x.dtype != torch.float32 or x.get_device() != c._device or x.dim() != 3 or x.shape[0] != n or \
            x.shape[1] != c._kv_heads or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor [{n}, {c._kv_heads}, rows] on cuda:{c._device}")
    return x.data_ptr(), x.shape[2]


def _decay(decay: Optional[float]) -> float:
    """The library's decay: below 0 where weights are left alone, which a caller says by None."""
    if decay is None:
        return -1.0
    if decay < 0:
        raise FmError(FM_ERR_INVALID_ARG, f"decay {decay}: at least 0, or None to leave the weights alone")
    return decay


def fm_kvq_create(n_layers: int, n_seqs: int, n_kv_heads: int, head_dim: int, max_rows: int,
                  stream=None) -> KvqCache:
    """An empty KV cache held in 4 bits, on the current device."""
    g = FmKvqConfig(n_layers, n_seqs, n_kv_heads, head_dim, max_rows)
    c = KvqCache()
    _kvq_check(load_library().fm_kvq_create(ctypes.byref(g), _stream(stream), ctypes.byref(c)))
    import torch
    c._kv_heads, c._head_dim, c._device = n_kv_heads, head_dim, torch.cuda.current_device()
    return c


def fm_kvq_append(c, layer: int, seq_ids: Sequence[int], k, v, n_rows: Sequence[int], starts: Sequence[int],
                  stream=None) -> None:
    """Rows k, v (CUDA tensors [sum(n_rows), n_kv_heads, head_dim], float32, float16 or bfloat16, packed in the order
    of seq_ids) become rows starts[i] .. of their sequences; each length is then starts[i] + n_rows[i]."""
    n, total = len(seq_ids), sum(n_rows)
    kp, dtype, _, ld = _kvq_rows(k, total, c._kv_heads, c, "k")
    vp, vt, _, vld = _kvq_rows(v, total, c._kv_heads, c, "v")
    if vt != dtype or vld != ld:
        raise ValueError("k and v differ in dtype or row stride")
    seq_ids_, n_rows_, starts_ = _ints(seq_ids, n, "seq_ids"), _ints(n_rows, n, "n_rows"), _ints(starts, n, "starts")
    _kvq_check(load_library().fm_kvq_append(c, layer, n, _addr(seq_ids_), _addr(n_rows_),
                                            _addr(starts_), kp, vp, dtype, ld, _stream(stream)), c)


def fm_kvq_read(c, layer: int, seq_ids: Sequence[int], rows: Sequence[int], n_rows: Sequence[int], k=None, v=None,
                weights=None, stream=None) -> None:
    """The values of rows rows[i] .. rows[i] + n_rows[i] - 1 into k and v (CUDA tensors [sum(n_rows), n_kv_heads,
    head_dim] or None), and their weights into weights (CUDA float32 [n_seqs, n_kv_heads, longest] or None)."""
    n, total = len(seq_ids), sum(n_rows)
    dtype, ld = FM_DTYPE_F32, c._kv_heads * c._head_dim
    kp = vp = None
    if k is not None:
        kp, dtype, _, ld = _kvq_rows(k, total, c._kv_heads, c, "k")
    if v is not None:
        vp, vt, _, vld = _kvq_rows(v, total, c._kv_heads, c, "v")
        if k is not None and (vt != dtype or vld != ld):
            raise ValueError("k and v differ in dtype or row stride")
        dtype, ld = vt, vld
    wp, ldw = _kvq_weights(weights, n, c, "weights")
    seq_ids_ = _ints(seq_ids, n, "seq_ids")
    rows_ = _ints(rows, n, "rows")
    n_rows_ = _ints(n_rows, n, "n_rows")
    _kvq_check(load_library().fm_kvq_read(c, layer, n, _addr(seq_ids_), _addr(rows_),
                                          _addr(n_rows_), kp, vp, dtype, ld, wp, ldw, _stream(stream)), c)


def fm_kvq_attend(c, layer: int, seq_ids: Sequence[int], q, n_rows: Sequence[int], out, scale: Optional[float] = None,
                  causal: bool = False, first_row: int = 0, decay: Optional[float] = None, weights=None,
                  stream=None) -> None:
    """Attention of n_rows[i] query rows of each sequence over its cache rows first_row .. (causal: the rows are the
    cache's last ones).  q, out: CUDA tensors [sum(n_rows), n_heads, head_dim] of one dtype (float32, float16,
    bfloat16); n_heads a multiple of n_kv_heads; scale: 1 / sqrt(head_dim) unless given.  decay: None leaves the
    rows' weights alone; a number d >= 0 counts them, w = d w + this call's, into weights too (CUDA float32 [n_seqs,
    n_kv_heads, rows] or None)."""
    n, total = len(seq_ids), sum(n_rows)
    qp, dtype, heads, ldq = _kvq_rows(q, total, None, c, "q")
    op, ot, _, ldo = _kvq_rows(out, total, heads, c, "out")
    if ot != dtype:
        raise ValueError("q and out differ in dtype")
    wp, ldw = _kvq_weights(weights, n, c, "weights")
    seq_ids_ = _ints(seq_ids, n, "seq_ids")
    n_rows_ = _ints(n_rows, n, "n_rows")
    _kvq_check(load_library().fm_kvq_attend(
        c, layer, n, _addr(seq_ids_), _addr(n_rows_), qp, dtype, heads, ldq,
        c._head_dim ** -0.5 if scale is None else scale, 1 if causal else 0, first_row, op, ldo,
        _decay(decay), wp, ldw, _stream(stream)), c)


def fm_kvq_set_weights(c, layer: int, seq_ids: Sequence[int], weights, stream=None) -> None:
    """The weights of each sequence's rows from a CUDA float32 tensor [n_seqs, n_kv_heads, >= longest]."""
    n = len(seq_ids)
    wp, ldw = _kvq_weights(weights, n, c, "weights")
    seq_ids_ = _ints(seq_ids, n, "seq_ids")
    _kvq_check(load_library().fm_kvq_set_weights(c, layer, n, _addr(seq_ids_), wp, ldw, _stream(stream)), c)


def fm_kvq_evict(c, layer: int, src_ids: Sequence[int], dst_ids: Sequence[int], keep: int, recent: int, kept=None,
                 stream=None) -> None:
    """Bring sequences down to keep rows a KV head: the last `recent` and, of the others, those of the largest weight.
    dst_ids[i] == src_ids[i] works in place.  kept: a contiguous CUDA int32 tensor [n_seqs, n_kv_heads, keep] that
    receives the rows kept, or None."""
    n = len(src_ids)
    if kept is not None:
        import torch
        if kept.dtype != torch.int32 or kept.get_device() != c._device or not kept.is_contiguous() or \
                tuple(kept.shape) != (n, c._kv_heads, keep):
            raise ValueError(f"kept must be a contiguous int32 tensor [{n}, {c._kv_heads}, {keep}] on cuda:{c._device}")
    src_ids_ = _ints(src_ids, n, "src_ids")
    dst_ids_ = _ints(dst_ids, n, "dst_ids")
    _kvq_check(load_library().fm_kvq_evict(c, layer, n, _addr(src_ids_), _addr(dst_ids_), keep,
                                           recent, _ptr(kept), _stream(stream)), c)


def fm_kvq_length(c, layer: int, seq: int) -> int:
    v = ctypes.c_int32()
    if load_library().fm_kvq_length(c, layer, seq, ctypes.byref(v)) != FM_OK:
        raise FmError(FM_ERR_INVALID_ARG, f"layer {layer}, sequence {seq}")
    return v.value


def fm_kvq_get_config(c) -> FmKvqConfig:
    g = FmKvqConfig()
    if load_library().fm_kvq_get_config(c, ctypes.byref(g)) != FM_OK:
        raise FmError(FM_ERR_INVALID_ARG, "no cache")
    return g


def fm_kvq_last_launch_count(c) -> int:
    n = ctypes.c_int32()
    _kvq_check(load_library().fm_kvq_last_launch_count(c, ctypes.byref(n)), c)
    return n.value


def fm_mtp_use_kvq(m, c, layer: int = 0, seq: int = 0, next_pos: Optional[int] = None,
                   decay: Optional[float] = None) -> None:
    """Keep the MTP head's rows in (layer, seq) of the 4-bit cache c (None: in its own f32 cache).  next_pos: the position
    after the cache's last row (its length unless given); decay: count the attention weights of every pass (None: do
    not).  The head keeps c alive while it uses it."""
    if c is not None and next_pos is None:
        next_pos = fm_kvq_length(c, layer, seq)
    _mtp_check(load_library().fm_mtp_use_kvq(m, c, layer, seq, next_pos or 0, _decay(decay)), m)
    m._kvq, m._paged = c, None


def fm_kvq_memory_bytes(c) -> int:
    v = ctypes.c_int64()
    _kvq_check(load_library().fm_kvq_memory_bytes(c, ctypes.byref(v)), c)
    return v.value


def fm_kvq_synchronize(c, stream=None) -> None:
    """Wait for the stream; raise FmError(FM_ERR_TIMEOUT) if a bounded device wait gave up since the last check."""
    _kvq_check(load_library().fm_kvq_synchronize(c, _stream(stream)), c)


def fm_kvq_selftest_wait_timeout(c, budget_us: int, stream=None) -> None:
    """Run a bounded device wait that cannot complete; it gives up after budget_us and the next fm_kvq_synchronize raises
    FmError(FM_ERR_TIMEOUT)."""
    _kvq_check(load_library().fm_kvq_selftest_wait_timeout(c, budget_us, _stream(stream)), c)


def fm_kvq_destroy(c) -> None:
    if c is not None and c.value:
        load_library().fm_kvq_destroy(c)
        c.value = None


class PagedCache(ctypes.c_void_p):
    """The handle of a paged KV cache; freed by fm_paged_destroy, or with the last reference to it.  Holds its pool."""

    def __del__(self):
        if self.value and _lib is not None:
            _lib.fm_paged_destroy(self)
            self.value = None


class PagedBatch:
    """A batch's place in a paged cache (fm_paged_batch); holds the tensors it was made from."""

    __slots__ = ("arg", "at", "tensors", "n_tokens", "workspace_bytes", "cache")


def _paged_check(status: int, c=None):
    if status != FM_OK:
        lib = load_library()
        raise FmError(status, f"{lib.fm_status_str(status).decode()}: {lib.fm_paged_last_error(c).decode()}")


def fm_paged_create(k_pool, v_pool, n_heads: int, rot_dims: int = 0, layout: int = FM_ROPE_INTERLEAVED, theta: float = 1e4,
                    scaling: int = FM_ROPE_PLAIN, factor: float = 1.0, original_rows: int = 0, low: float = 1.0,
                    high: float = 32.0, gain: float = 1.0, eps: float = 1e-6, stream=None) -> PagedCache:
    """A KV cache in pages over the caller's pool: k_pool, v_pool, contiguous CUDA tensors [n_layers, n_pages, n_kv_heads,
    page_rows, head_dim] of float16 or bfloat16, on the current device.  n_heads query heads read it.  The first rot_dims
    of a head are rotated by position in `layout`'s pairs, the angles scaled as `scaling` says."""
    import torch
    dtypes = {torch.float16: FM_DTYPE_F16, torch.bfloat16: FM_DTYPE_BF16}
    if k_pool.dtype not in dtypes or v_pool.dtype != k_pool.dtype or v_pool.shape != k_pool.shape or k_pool.dim() != 5:
        raise ValueError("k_pool and v_pool must be float16 or bfloat16 tensors [layers, pages, kv_heads, page_rows, head_dim] of "
                         "one shape and dtype")
    if not (k_pool.is_cuda and k_pool.is_contiguous() and v_pool.is_contiguous()) or v_pool.device != k_pool.device:
        raise ValueError("k_pool and v_pool must be contiguous and on one CUDA device")
    if k_pool.get_device() != torch.cuda.current_device():
        raise ValueError(f"the pool is on cuda:{k_pool.get_device()}, the current device is cuda:{torch.cuda.current_device()}")
    layers, pages, kv_heads, page_rows, head_dim = k_pool.shape
    g = FmPagedConfig(layers, pages, page_rows, n_heads, kv_heads, head_dim, dtypes[k_pool.dtype], rot_dims, layout, scaling,
                      original_rows, theta, factor, low, high, gain, eps)
    c = PagedCache()
    _paged_check(load_library().fm_paged_create(ctypes.byref(g), k_pool.data_ptr(), v_pool.data_ptr(), _stream(stream),
                                                ctypes.byref(c)))
    c._pool, c._heads, c._kv_heads, c._head_dim = (k_pool, v_pool), n_heads, kv_heads, head_dim
    c._dtype, c._code, c._device, c._f32 = k_pool.dtype, dtypes[k_pool.dtype], k_pool.get_device(), torch.float32
    empty, uint8, device = torch.empty, torch.uint8, k_pool.device
    c._workspace = lambda n: empty(n, dtype=uint8, device=device)
    return c


def fm_paged_batch(c, starts, lengths, table, n_tokens: int, max_new: Optional[int] = None) -> PagedBatch:
    """The place of a batch's new rows: starts [n_seqs + 1], lengths [n_seqs] and table [n_seqs, pages], int32 CUDA tensors
    whose values the calls read when they run (so they may be rewritten in place, between a graph's replays too).  n_tokens:
    packed rows; max_new: the most new rows a sequence may have (n_tokens unless given)."""
    import torch
    n = lengths.shape[0]
    for x, what, shape in ((starts, "starts", (n + 1,)), (lengths, "lengths", (n,)), (table, "table", (n, table.shape[-1]))):
        if x.dtype != torch.int32 or x.get_device() != c._device or tuple(x.shape) != shape:
            raise ValueError(f"{what} must be an int32 tensor {list(shape)} on cuda:{c._device}")
        if x.numel() and x.shape[-1] > 1 and x.stride(-1) != 1:
            raise ValueError(f"{what} must be contiguous along its last axis")
    b = PagedBatch()
    ld = table.stride(0) if n > 1 else table.shape[1]
    b.arg = FmPagedBatch(starts.data_ptr(), lengths.data_ptr(), table.data_ptr(), ld, n, n_tokens, table.shape[1],
                         n_tokens if max_new is None else max_new)
    b.at, b.tensors, b.n_tokens, b.cache = ctypes.addressof(b.arg), (starts, lengths, table), n_tokens, c
    b.workspace_bytes = fm_paged_workspace_bytes(c, b.arg.max_new)
    return b


def _paged_rows(x, heads: int, n_tokens: int, c, dtype, what: str) -> array.array:
    """The library's view (an fm_paged_rows; a quarter of the time that a ctypes structure takes) of a tensor [>= n_tokens,
    heads, head_dim] whose last axis is contiguous."""
    if x.dtype is not dtype or x.get_device() != c._device:
        raise ValueError(f"{what} must be a {dtype} tensor on cuda:{c._device}")
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[0] < n_tokens or shape[1] != heads or shape[2] != c._head_dim:
        raise ValueError(f"{what} has shape {tuple(shape)}, expected [{n_tokens}, {heads}, {c._head_dim}]")
    if stride[2] != 1:
        raise ValueError(f"{what}: a row's values must be contiguous")
    return array.array("q", (x.data_ptr(), stride[0], stride[1]))


def _paged_norm(w, c, what: str):
    if w is None:
        return None
    if w.dtype is not c._f32 or w.get_device() != c._device or w.shape != (c._head_dim,) or not w.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor [{c._head_dim}] on cuda:{c._device}")
    return w.data_ptr()


def fm_paged_write(c, layer: int, batch: PagedBatch, q=None, k=None, v=None, q_out=None, q_norm=None, k_norm=None,
                   stream=None) -> None:
    """The batch's new rows into the pages of `layer`: k (normed by k_norm, rotated) and v, and q (normed by q_norm, rotated)
    into q_out.  q: [n_tokens, n_heads, head_dim], k, v: [n_tokens, n_kv_heads, head_dim], of float32 or the pool's type, any
    stride between tokens and heads (whole 16 bytes); q_out: of the pool's type.  q and q_out, or k and v, may be None;
    norms: float32 [head_dim] or None."""
    if batch.cache is not c:
        raise ValueError("the batch was made for another cache")
    first, n = q if q is not None else k, batch.n_tokens
    t = c._f32 if first is not None and first.dtype is c._f32 else c._dtype
    q_ = None if q is None else _paged_rows(q, c._heads, n, c, t, "q")
    k_ = None if k is None else _paged_rows(k, c._kv_heads, n, c, t, "k")
    v_ = None if v is None else _paged_rows(v, c._kv_heads, n, c, t, "v")
    o_ = None if q_out is None else _paged_rows(q_out, c._heads, n, c, c._dtype, "q_out")
    _paged_check(_lib.fm_paged_write(
        c, layer, batch.at, None if q_ is None else _addr(q_), None if k_ is None else _addr(k_), None if v_ is None else _addr(v_),
        FM_DTYPE_F32 if t is c._f32 else c._code, _paged_norm(q_norm, c, "q_norm"), _paged_norm(k_norm, c, "k_norm"),
        None if o_ is None else _addr(o_), _stream(stream)), c)


def fm_paged_attend(c, layer: int, batch: PagedBatch, q, out, scale: Optional[float] = None, causal: bool = True, window: int = 0,
                    sinks: int = 0, workspace=None, stream=None) -> None:
    """Attention of the batch's new rows over the pages of `layer`; q, out: [n_tokens, n_heads, head_dim] of the pool's type.
    scale: 1 / sqrt(head_dim) unless given; window: rows a row sees back from its own (0: all), and the first `sinks` rows
    besides.  workspace: a CUDA uint8 tensor of at least batch.workspace_bytes that nothing else uses until the call is done;
    one is allocated in the call's stream (or the graph's pool) unless given."""
    if batch.cache is not c:
        raise ValueError("the batch was made for another cache")
    size = batch.workspace_bytes
    if workspace is None:
        if stream is None:
            workspace = c._workspace(size)
        else:
            import torch
            other = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream), device=q.device)
            with torch.cuda.stream(other):
                workspace = c._workspace(size)
    elif workspace.get_device() != c._device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{c._device}")
    else:
        size = workspace.nbytes
    n = batch.n_tokens
    q_ = _paged_rows(q, c._heads, n, c, c._dtype, "q")
    o_ = _paged_rows(out, c._heads, n, c, c._dtype, "out")
    _paged_check(_lib.fm_paged_attend(
        c, layer, batch.at, _addr(q_), _addr(o_), c._head_dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, sinks,
        workspace.data_ptr(), size, _stream(stream)), c)


def fm_paged_workspace_bytes(c, max_new: int) -> int:
    v = ctypes.c_int64()
    _paged_check(load_library().fm_paged_workspace_bytes(c, max_new, ctypes.byref(v)), c)
    return v.value


def fm_paged_get_config(c) -> FmPagedConfig:
    g = FmPagedConfig()
    _paged_check(load_library().fm_paged_get_config(c, ctypes.byref(g)), c)
    return g


def fm_paged_last_launch_count(c) -> int:
    n = ctypes.c_int32()
    _paged_check(load_library().fm_paged_last_launch_count(c, ctypes.byref(n)), c)
    return n.value


def fm_paged_synchronize(c, stream=None) -> None:
    """Wait for the stream; raise FmError(FM_ERR_TIMEOUT) if a bounded device wait gave up, FmError(FM_ERR_INVALID_ARG) if a
    batch's starts, lengths or pages pointed outside, since the last check.  Where both happened, the next call raises the
    second."""
    _paged_check(load_library().fm_paged_synchronize(c, _stream(stream)), c)


def fm_paged_selftest_wait_timeout(c, budget_us: int, stream=None) -> None:
    """Run a bounded device wait that cannot complete; it gives up after budget_us and the next fm_paged_synchronize raises
    FmError(FM_ERR_TIMEOUT)."""
    _paged_check(load_library().fm_paged_selftest_wait_timeout(c, budget_us, _stream(stream)), c)


def fm_paged_destroy(c) -> None:
    if c is not None and c.value:
        load_library().fm_paged_destroy(c)
        c.value = None
        c._pool = None


def fm_mtp_use_paged(m, c, layer: int = 0, table=None, window: int = 0, sinks: int = 0) -> None:
    """Keep the MTP head's rows in `layer` of the paged cache c (None: in its own f32 cache).  table: a contiguous CUDA int32
    tensor [pages], the pages of the head's sequence; window, sinks: as fm_paged_attend's.  The head keeps c and table alive
    while it uses them."""
    if c is not None:
        import torch
        if table is None or table.dtype != torch.int32 or table.get_device() != c._device or table.dim() != 1 or \
                not table.is_contiguous():
            raise ValueError(f"table must be a contiguous int32 tensor [pages] on cuda:{c._device}")
    _mtp_check(load_library().fm_mtp_use_paged(m, c, layer, _ptr(table) if c is not None else None,
                                               table.shape[0] if c is not None else 0, window, sinks), m)
    m._paged, m._kvq = None if c is None else (c, table), None
