"""Python binding of the GB300 per-step multi-codebook token sampler.

Thin ctypes marshalling over the C ABI in ``include/ts_sampler.h``; every step
of sampling runs in the CUDA kernels of ``libts_sampler.so``.  PyTorch is used
only for device memory and streams.  The functions keep the C names:

    ts_create, ts_destroy, ts_max_top_k, ts_sample, ts_sample_debug,
    ts_sample_steps, ts_reserve, ts_sample_noalloc, ts_advance_steps,
    ts_read_status, ts_set_option, ts_plan, ts_status_string, ts_last_error,
    ts_lm_head_logits, ts_lm_head_sample, ts_sample_host,
    ts_reserve_kv, ts_kv_tables, ts_kv_append, ts_paged_attention,
    ts_kv_debug_lose_parts,
    ts_rms_norm, ts_gate, ts_linear_e4m3, ts_rotary, ts_kv_append_rotary,
    ts_rotary_frequencies

``Sampler`` wraps a handle; ``DeviceBatch`` holds one step's per-row arrays on
the GPU with a prebuilt ``ts_batch`` so that repeated calls marshal nothing;
``LmHead`` holds a frame's hidden states and output heads with a prebuilt
``ts_lm_head``; ``KvTables``, ``KvCache``, ``KvTokens`` and ``PagedQuery`` do the
same for the paged key-value cache's calls, ``RmsNorm``, ``Gate``,
``LinearE4m3`` and ``Rotary`` for the layer operators around it.
Importing this module loads the compiled library and raises if it is missing;
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

from . import _build

TS_OK = 0
TS_ERR_INVALID_ARG = 1
TS_ERR_UNSUPPORTED = 2
TS_ERR_CUDA = 3
TS_ERR_NO_MEMORY = 4
TS_DTYPE_F32 = 0
TS_DTYPE_BF16 = 1
TS_DTYPE_E4M3 = 2
TS_ROW_BAD_SHAPE = 1
TS_ROW_BAD_PARAM = 2
TS_ROW_NONFINITE = 4
TS_ROW_BAD_SLOT = 8
TS_ROW_NOT_READY = 16
TS_ROW_BAD_BLOCK = 32
TS_ROW_NO_BLOCKS = 64
TS_ROW_STALLED = 128
TS_OPT_PATH = 1
TS_OPT_CLUSTER = 2
TS_OPT_PDL = 3
TS_OPT_WIDE_EXACT = 4
TS_OPT_WARPS_PER_ROW = 5
TS_OPT_FAIL_LAUNCH = 6
TS_OPT_KV_CTAS = 7
TS_OPT_KV_JOIN = 8
TS_OPT_LINEAR_SPLIT = 9
TS_OPT_LINEAR_PATH = 10
TS_OPT_LINEAR_SHARE = 11
TS_OPT_LINEAR_LOSE = 12
TS_MAX_VOCAB_BF16 = 163840
TS_MAX_VOCAB_F32 = 81920
TS_NOALLOC_SCRATCH_BYTES = 4194304
TS_NOALLOC_MAX_ROWS = 64
TS_LM_HEAD_DIM_STEP = 64
TS_LM_HEAD_MAX_DIM = 16384
TS_KV_MAX_REQUESTS = 8192
TS_KV_MAX_LEN = 2147482624
TS_KV_MAX_HEAD_DIM = 256
TS_KV_MAX_HEADS = 65536
TS_SCALE_BLOCK = 128
TS_NORM_MAX_DIM = 32768
TS_GATE_MAX_DIM = 1048576
TS_LINEAR_MAX_DIM = 1048576
TS_LINEAR_MAX_ROWS = 2147482624
TS_ROTARY_MAX_HEAD_DIM = 1024
TS_ACT_NONE = 0
TS_ACT_SILU = 1
TS_ACT_GELU = 2
TS_ACT_GELU_TANH = 3
TS_ROPE_PLAIN = 0
TS_ROPE_LINEAR = 1
TS_ROPE_NTK = 2
TS_ROPE_BY_PARTS = 3

EXPORTED = ("ts_create", "ts_destroy", "ts_max_top_k", "ts_sample", "ts_sample_debug",
            "ts_sample_steps", "ts_reserve", "ts_sample_noalloc", "ts_advance_steps",
            "ts_read_status", "ts_set_option", "ts_plan", "ts_status_string", "ts_last_error",
            "ts_lm_head_logits", "ts_lm_head_sample", "ts_sample_host",
            "ts_reserve_kv", "ts_kv_tables", "ts_kv_append", "ts_paged_attention",
             "ts_kv_debug_lose_parts",
            "ts_rms_norm", "ts_gate", "ts_linear_e4m3", "ts_rotary", "ts_kv_append_rotary",
            "ts_rotary_frequencies")


class TsBatch(ctypes.Structure):
    """Mirror of ``ts_batch``."""
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("logits_len", ctypes.c_int64),
        ("n_rows", ctypes.c_int32),
        ("max_row_vocab", ctypes.c_int32),
        ("row_vocab", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p),
        ("temp", ctypes.c_void_p),
        ("top_k", ctypes.c_void_p),
        ("top_p", ctypes.c_void_p),
        ("seed", ctypes.c_void_p),
        ("request", ctypes.c_void_p),
        ("codebook", ctypes.c_void_p),
        ("row_stream", ctypes.c_void_p),
        ("step", ctypes.c_void_p),
        ("n_streams", ctypes.c_int32),
        ("eos_id", ctypes.c_void_p),
        ("out_ids", ctypes.c_void_p),
        ("out_eos", ctypes.c_void_p),
        ("feedback_buf", ctypes.c_void_p),
        ("feedback_slot", ctypes.c_void_p),
        ("feedback_len", ctypes.c_int64),
        ("advance_steps", ctypes.c_int32),
        ("stop_step", ctypes.c_void_p),
        ("max_steps", ctypes.c_void_p),
        ("finish_reason", ctypes.c_void_p),
        ("pad_id", ctypes.c_int32),
        ("hist_ring", ctypes.c_void_p),
        ("hist_len", ctypes.c_int32),
        ("hist_codebooks", ctypes.c_int32),
        ("rep_penalty", ctypes.c_void_p),
        ("step_out", ctypes.c_void_p),
    ]


class TsSteps(ctypes.Structure):
    """Mirror of ``ts_steps``."""
    _fields_ = [
        ("n_steps", ctypes.c_int32),
        ("logits_step_stride", ctypes.c_int64),
        ("out_step_stride", ctypes.c_int64),
        ("feedback_step_stride", ctypes.c_int64),
        ("ready", ctypes.c_void_p),
        ("ready_timeout_ns", ctypes.c_uint64),
    ]


class TsLmHead(ctypes.Structure):
    """Mirror of ``ts_lm_head``."""
    _fields_ = [
        ("hidden", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("weights_len", ctypes.c_int64),
        ("head_offsets", ctypes.c_void_p),
        ("dim", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
    ]


class TsKvTables(ctypes.Structure):
    """Mirror of ``ts_kv_tables_args``."""
    _fields_ = [
        ("n_requests", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("n_blocks", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32),
        ("table_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("lens", ctypes.c_void_p),
        ("lens_out", ctypes.c_void_p),
        ("n_new", ctypes.c_void_p),
        ("finished", ctypes.c_void_p),
        ("free_blocks", ctypes.c_void_p),
        ("free_len", ctypes.c_int32),
        ("n_free", ctypes.c_void_p),
        ("n_free_out", ctypes.c_void_p),
        ("max_tokens", ctypes.c_int32),
        ("token_starts", ctypes.c_void_p),
        ("slots", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("requests", ctypes.c_void_p),
    ]


class TsKvCache(ctypes.Structure):
    """Mirror of ``ts_kv_cache``."""
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("n_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("k_block_stride", ctypes.c_int64),
        ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_block_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]


class TsKvTokens(ctypes.Structure):
    """Mirror of ``ts_kv_tokens``."""
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("n_tokens", ctypes.c_int32),
        ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("slots", ctypes.c_void_p),
        ("rows", ctypes.c_void_p),
        ("n_rows", ctypes.c_int32),
    ]


class TsPagedQuery(ctypes.Structure):
    """Mirror of ``ts_paged_query``."""
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("n_requests", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32),
        ("q_request_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("out_request_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64),
        ("lens", ctypes.c_void_p),
        ("key_mask", ctypes.c_void_p),
        ("mask_stride", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("window", ctypes.c_int32),
    ]


class TsNorm(ctypes.Structure):
    """Mirror of ``ts_norm_args``."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("residual", ctypes.c_void_p),
        ("residual_out", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("out_scale", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("n_rows", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("x_stride", ctypes.c_int64),
        ("residual_stride", ctypes.c_int64),
        ("residual_out_stride", ctypes.c_int64),
        ("out_stride", ctypes.c_int64),
        ("out_scale_stride", ctypes.c_int64),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
    ]


class TsGate(ctypes.Structure):
    """Mirror of ``ts_gate_args``."""
    _fields_ = [
        ("up", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("out_scale", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("n_rows", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("up_stride", ctypes.c_int64),
        ("gate_stride", ctypes.c_int64),
        ("out_stride", ctypes.c_int64),
        ("out_scale_stride", ctypes.c_int64),
    ]


class TsLinear(ctypes.Structure):
    """Mirror of ``ts_linear_args``."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("x_scale", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("w_scale", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("out_dtype", ctypes.c_int32),
        ("n_rows", ctypes.c_int32),
        ("in_dim", ctypes.c_int32),
        ("out_dim", ctypes.c_int32),
        ("x_stride", ctypes.c_int64),
        ("x_scale_stride", ctypes.c_int64),
        ("w_stride", ctypes.c_int64),
        ("w_scale_stride", ctypes.c_int64),
        ("out_stride", ctypes.c_int64),
    ]


class TsRotary(ctypes.Structure):
    """Mirror of ``ts_rotary_args``."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("n_tokens", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("x_token_stride", ctypes.c_int64),
        ("x_head_stride", ctypes.c_int64),
        ("out_token_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("positions", ctypes.c_void_p),
        ("rows", ctypes.c_void_p),
        ("n_rows", ctypes.c_int32),
        ("amplitude", ctypes.c_float),
        ("freqs", ctypes.c_void_p),
    ]


class SamplerError(RuntimeError):
    def __init__(self, status: int, what: str):
        detail = _lib.ts_last_error().decode() if status == TS_ERR_CUDA else ""
        msg = f"{what}: {_lib.ts_status_string(status).decode()}"
        super().__init__(msg + (f" ({detail})" if detail else ""))
        self.status = status


def _load(path: str):
    if not os.path.exists(path):
        raise ImportError(f"sampler library not built: {path} (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "ts_create": ([ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)], ctypes.c_int),
        "ts_destroy": ([vp], ctypes.c_int),
        "ts_max_top_k": ([vp], i32),
        "ts_sample": ([vp, ctypes.POINTER(TsBatch), vp], ctypes.c_int),
        "ts_sample_debug": ([vp, ctypes.POINTER(TsBatch), i32, vp, vp, vp, vp, vp], ctypes.c_int),
        "ts_sample_steps": ([vp, ctypes.POINTER(TsBatch), ctypes.POINTER(TsSteps), vp],
                            ctypes.c_int),
        "ts_reserve": ([vp, i32, i32], ctypes.c_int),
        "ts_sample_noalloc": ([i32, ctypes.POINTER(TsBatch), vp, vp], ctypes.c_int),
        "ts_advance_steps": ([vp, i32, vp], ctypes.c_int),
        "ts_read_status": ([vp, ctypes.POINTER(ctypes.c_uint32), vp], ctypes.c_int),
        "ts_set_option": ([vp, i32, i32], ctypes.c_int),
        "ts_plan": ([vp, ctypes.POINTER(TsBatch)] + [ctypes.POINTER(i32)] * 5, ctypes.c_int),
        "ts_sample_host": ([vp, ctypes.POINTER(TsBatch), vp, vp, vp, vp], ctypes.c_int),
        "ts_lm_head_logits": ([vp, ctypes.POINTER(TsLmHead), ctypes.POINTER(TsBatch), vp],
                              ctypes.c_int),
        "ts_lm_head_sample": ([vp, ctypes.POINTER(TsLmHead), ctypes.POINTER(TsBatch), vp],
                              ctypes.c_int),
        "ts_reserve_kv": ([vp, i32], ctypes.c_int),
        "ts_kv_tables": ([vp, ctypes.POINTER(TsKvTables), vp], ctypes.c_int),
        "ts_kv_append": ([vp, ctypes.POINTER(TsKvCache), ctypes.POINTER(TsKvTokens), vp],
                         ctypes.c_int),
        "ts_paged_attention": ([vp, ctypes.POINTER(TsKvCache), ctypes.POINTER(TsPagedQuery), vp],
                               ctypes.c_int),
        "ts_kv_debug_lose_parts": ([vp, i32], ctypes.c_int),
        "ts_rms_norm": ([vp, ctypes.POINTER(TsNorm), vp], ctypes.c_int),
        "ts_gate": ([vp, ctypes.POINTER(TsGate), vp], ctypes.c_int),
        "ts_linear_e4m3": ([vp, ctypes.POINTER(TsLinear), vp], ctypes.c_int),
        "ts_rotary": ([vp, ctypes.POINTER(TsRotary), vp], ctypes.c_int),
        "ts_kv_append_rotary": ([vp, ctypes.POINTER(TsKvCache), ctypes.POINTER(TsKvTokens),
                                 ctypes.POINTER(TsRotary), vp], ctypes.c_int),
        "ts_rotary_frequencies": ([vp, i32] + [ctypes.c_double, i32] + [ctypes.c_double] * 4
                                  + [ctypes.POINTER(ctypes.c_float)], ctypes.c_int),
        "ts_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "ts_last_error": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    del i64
    return lib


LIB_PATH = _build.LIB_PATH
_lib = _load(LIB_PATH)


def library():
    """The loaded ctypes library (for symbol checks)."""
    return _lib


def _check(status: int, what: str):
    if status != TS_OK:
        raise SamplerError(status, what)


_current_stream = None  # () -> the current stream's address


def _stream_ptr(stream) -> int:
    global _current_stream
    if stream is not None:
        return int(stream.cuda_stream)
    if _current_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:  # without a Stream object per call
            _current_stream = lambda: raw(torch.cuda.current_device())  # noqa: E731
        else:
            _current_stream = lambda: int(torch.cuda.current_stream().cuda_stream)  # noqa: E731
    return _current_stream()


# --------------------------------------------------------------------------
# C-named functions
# --------------------------------------------------------------------------
def ts_create(device: int = 0, max_top_k: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(_lib.ts_create(device, max_top_k, ctypes.byref(h)), "ts_create")
    return h.value


def ts_destroy(handle: int) -> None:
    _check(_lib.ts_destroy(handle), "ts_destroy")


def ts_max_top_k(handle: int) -> int:
    return int(_lib.ts_max_top_k(handle))


def ts_sample(handle: int, batch: "DeviceBatch", stream=None) -> None:
    _check(_lib.ts_sample(handle, ctypes.byref(batch.c), _stream_ptr(stream)), "ts_sample")


def ts_sample_debug(handle: int, batch: "DeviceBatch", max_keep: int, kept_ids, kept_probs,
                    n_kept, n_nucleus, stream=None) -> None:
    _check(_lib.ts_sample_debug(handle, ctypes.byref(batch.c), max_keep, kept_ids.data_ptr(),
                                kept_probs.data_ptr(), n_kept.data_ptr(), n_nucleus.data_ptr(),
                                _stream_ptr(stream)), "ts_sample_debug")


def ts_sample_steps(handle: int, batch: "DeviceBatch", steps: TsSteps, stream=None) -> None:
    _check(_lib.ts_sample_steps(handle, ctypes.byref(batch.c), ctypes.byref(steps),
                                _stream_ptr(stream)), "ts_sample_steps")


def ts_reserve(handle: int, max_rows: int, max_row_vocab: int) -> None:
    _check(_lib.ts_reserve(handle, max_rows, max_row_vocab), "ts_reserve")


def ts_sample_noalloc(batch: "DeviceBatch", max_top_k: int = 0, status=None,
                      stream=None) -> None:
    """Samples ``batch`` without any allocation, for callers whose memory is
    all owned by their own pool (the workspace is the library's static scratch
    array).  ``status``: a one-element int32 device tensor that collects the
    row error bits, or None."""
    st = _lib.ts_sample_noalloc(max_top_k, ctypes.byref(batch.c),
                                status.data_ptr() if status is not None else None,
                                _stream_ptr(stream))
    if st == TS_ERR_UNSUPPORTED:
        raise SamplerError(st, f"ts_sample_noalloc ({ts_last_error()})")
    _check(st, "ts_sample_noalloc")


def ts_advance_steps(step, stream=None) -> None:
    _check(_lib.ts_advance_steps(step.data_ptr(), step.numel(), _stream_ptr(stream)),
           "ts_advance_steps")


def ts_read_status(handle: int, stream=None) -> int:
    bits = ctypes.c_uint32()
    _check(_lib.ts_read_status(handle, ctypes.byref(bits), _stream_ptr(stream)), "ts_read_status")
    return int(bits.value)


def ts_set_option(handle: int, option: int, value: int) -> None:
    _check(_lib.ts_set_option(handle, option, value), "ts_set_option")


def ts_plan(handle: int, batch: "DeviceBatch") -> dict:
    out = [ctypes.c_int32() for _ in range(5)]
    _check(_lib.ts_plan(handle, ctypes.byref(batch.c), *[ctypes.byref(o) for o in out]),
           "ts_plan")
    keys = ("path", "ctas_per_row", "threads", "smem_bytes", "grid")
    return {k: int(o.value) for k, o in zip(keys, out)}


def ts_sample_host(handle: int, batch: "DeviceBatch", host_logits, host_ids, host_eos,
                   stream=None) -> None:
    """Host logits in, host ids and EOS flags out (see the header).  The
    three host buffers are CPU tensors (pinned for asynchronous copies) or
    numpy arrays: logits in the batch's layout (int16 / uint16 bits for bf16,
    float32), int32 ids and uint8 flags of n_rows each."""
    def ptr(a):
        return a.data_ptr() if hasattr(a, "data_ptr") else a.ctypes.data
    _check(_lib.ts_sample_host(handle, ctypes.byref(batch.c), ptr(host_logits), ptr(host_ids),
                               ptr(host_eos), _stream_ptr(stream)), "ts_sample_host")


def ts_lm_head_logits(handle: int, head: "LmHead", batch: "DeviceBatch", stream=None) -> None:
    _check(_lib.ts_lm_head_logits(handle, ctypes.byref(head.c), ctypes.byref(batch.c),
                                  _stream_ptr(stream)), "ts_lm_head_logits")


def ts_lm_head_sample(handle: int, head: "LmHead", batch: "DeviceBatch", stream=None) -> None:
    _check(_lib.ts_lm_head_sample(handle, ctypes.byref(head.c), ctypes.byref(batch.c),
                                  _stream_ptr(stream)), "ts_lm_head_sample")


def ts_reserve_kv(handle: int, max_requests: int) -> None:
    """The workspace of the paged cache's calls: once, before any capture."""
    _check(_lib.ts_reserve_kv(handle, max_requests), "ts_reserve_kv")


def ts_kv_tables(handle: int, tables: "KvTables", stream=None) -> None:
    """Block tables, lengths and slot maps of the next tokens (see the header)."""
    _check(_lib.ts_kv_tables(handle, ctypes.byref(tables.c), _stream_ptr(stream)), "ts_kv_tables")


def ts_kv_append(handle: int, cache: "KvCache", tokens: "KvTokens", stream=None) -> None:
    """Writes the tokens' keys and values into the cache at their slots; they have
    its heads, row width and device (ValueError)."""
    if tokens.rows_of != cache.rows_of:
        raise ValueError(f"tokens of {tokens.rows_of} for a cache of {cache.rows_of}")
    _check(_lib.ts_kv_append(handle, ctypes.byref(cache.c), ctypes.byref(tokens.c),
                             _stream_ptr(stream)), "ts_kv_append")


def ts_paged_attention(handle: int, cache: "KvCache", query: "PagedQuery", stream=None) -> None:
    """Attention of one query token per request over its cached tokens; queries
    have the cache's row width and device, a key mask a column for each token of a
    table row (ValueError)."""
    if query.rows_of != cache.rows_of[1:]:
        raise ValueError(f"queries of {query.rows_of} for a cache of {cache.rows_of[1:]}")
    if query.key_mask is not None:
        tokens = query.block_table.shape[1] * cache.k.shape[1]
        if query.key_mask.shape[1] < tokens:
            raise ValueError(f"key_mask: {query.key_mask.shape[1]} columns for tables of {tokens} tokens")
    _check(_lib.ts_paged_attention(handle, ctypes.byref(cache.c), ctypes.byref(query.c),
                                   _stream_ptr(stream)), "ts_paged_attention")


def ts_kv_debug_lose_parts(handle: int, come: int) -> None:
    """For tests: the workspace's counters as a call leaves them that lost parts."""
    _check(_lib.ts_kv_debug_lose_parts(handle, come), "ts_kv_debug_lose_parts")


def ts_rms_norm(handle: int, norm: "RmsNorm", stream=None) -> None:
    """The residual's sum, its root-mean-square norm and 8-bit rows of it (see the header)."""
    _check(_lib.ts_rms_norm(handle, ctypes.byref(norm.c), _stream_ptr(stream)), "ts_rms_norm")


def ts_gate(handle: int, gate: "Gate", stream=None) -> None:
    """A gated activation, or only the rounding to 8-bit rows (see the header)."""
    _check(_lib.ts_gate(handle, ctypes.byref(gate.c), _stream_ptr(stream)), "ts_gate")


def ts_linear_e4m3(handle: int, linear: "LinearE4m3", stream=None) -> None:
    """The product of 8-bit rows and 8-bit weights with block scales (see the header)."""
    _check(_lib.ts_linear_e4m3(handle, ctypes.byref(linear.c), _stream_ptr(stream)), "ts_linear_e4m3")


def ts_rotary(handle: int, rotary: "Rotary", stream=None) -> None:
    """Rotary positions of one tensor's heads (see the header)."""
    _check(_lib.ts_rotary(handle, ctypes.byref(rotary.c), _stream_ptr(stream)), "ts_rotary")


def ts_kv_append_rotary(handle: int, cache: "KvCache", tokens: "KvTokens", rotary: "Rotary",
                        stream=None) -> None:
    """``ts_rotary`` of the queries and ``ts_kv_append`` of the same tokens, whose keys
    are turned alike, in one launch.  Tokens have the cache's heads, row width and
    device, queries its row width and device (ValueError)."""
    if tokens.rows_of != cache.rows_of:
        raise ValueError(f"tokens of {tokens.rows_of} for a cache of {cache.rows_of}")
    if rotary.rows_of != cache.rows_of[1:]:
        raise ValueError(f"queries of {rotary.rows_of} for a cache of {cache.rows_of[1:]}")
    _check(_lib.ts_kv_append_rotary(handle, ctypes.byref(cache.c), ctypes.byref(tokens.c),
                                    ctypes.byref(rotary.c), _stream_ptr(stream)), "ts_kv_append_rotary")


def ts_rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: int = TS_ROPE_PLAIN, *,
                          factor: float = 1.0, original_len: float = 1.0, low: float = 1.0,
                          high: float = 32.0):
    """The frequencies that ``Rotary`` takes, as a float64 array on the host, and the
    amplitude that belongs to them (see the header)."""
    _need(0 < rotary_dim <= TS_ROTARY_MAX_HEAD_DIM, "rotary_dim: from 2 to a head's largest width")
    freqs = np.zeros(max(1, rotary_dim // 2), np.float64)
    amplitude = ctypes.c_float()
    _check(_lib.ts_rotary_frequencies(freqs.ctypes.data, rotary_dim, base, scaling, factor, original_len,
                                      low, high, ctypes.byref(amplitude)), "ts_rotary_frequencies")
    return freqs, float(amplitude.value)


def ts_status_string(status: int) -> str:
    return _lib.ts_status_string(status).decode()


def ts_last_error() -> str:
    return _lib.ts_last_error().decode()


# --------------------------------------------------------------------------
# Convenience wrappers
# --------------------------------------------------------------------------
class Sampler:
    """Owns a ``ts_sampler`` handle on one device."""

    def __init__(self, device: int = 0, max_top_k: int = 0):
        self.handle = ts_create(device, max_top_k)
        self.device = device

    @property
    def cap(self) -> int:
        return ts_max_top_k(self.handle)

    def sample(self, batch: "DeviceBatch", stream=None) -> None:
        ts_sample(self.handle, batch, stream)

    def reserve_kv(self, max_requests: int) -> None:
        ts_reserve_kv(self.handle, max_requests)

    def sample_debug(self, batch: "DeviceBatch", max_keep: int, stream=None) -> dict:
        import torch
        n = batch.n_rows
        dev = batch.out_ids.device
        kept_ids = torch.full((n, max_keep), -1, dtype=torch.int32, device=dev)
        kept_probs = torch.zeros((n, max_keep), dtype=torch.float32, device=dev)
        n_kept = torch.zeros(n, dtype=torch.int32, device=dev)
        n_nucleus = torch.zeros(n, dtype=torch.int32, device=dev)
        ts_sample_debug(self.handle, batch, max_keep, kept_ids, kept_probs, n_kept, n_nucleus,
                        stream)
        return {"kept_ids": kept_ids, "kept_probs": kept_probs, "n_kept": n_kept,
                "n_nucleus": n_nucleus}

    def sample_steps(self, batch: "DeviceBatch", n_steps: int, *, logits_step_stride: int,
                     out_step_stride: int, feedback_step_stride: int = 0, ready=None,
                     ready_timeout_ns: int = 0, stream=None) -> None:
        """``n_steps`` decode steps of ``batch`` in one launch (see ts_sample_steps);
        ``ready``: a uint32/int32 tensor of per-step flags the device can read, or None."""
        st = TsSteps()
        st.n_steps = n_steps
        st.logits_step_stride = logits_step_stride
        st.out_step_stride = out_step_stride
        st.feedback_step_stride = feedback_step_stride
        st.ready = ready.data_ptr() if ready is not None else None
        st.ready_timeout_ns = ready_timeout_ns
        ts_sample_steps(self.handle, batch, st, stream)

    def read_status(self, stream=None) -> int:
        return ts_read_status(self.handle, stream)

    def reserve(self, max_rows: int, max_row_vocab: int) -> None:
        ts_reserve(self.handle, max_rows, max_row_vocab)

    def set_option(self, option: int, value: int) -> None:
        ts_set_option(self.handle, option, value)

    def plan(self, batch: "DeviceBatch") -> dict:
        return ts_plan(self.handle, batch)

    def close(self) -> None:
        if getattr(self, "handle", None):
            ts_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_ARRAYS = (("row_vocab", np.int32), ("row_offsets", np.int64), ("temp", np.float32),
           ("top_k", np.int32), ("top_p", np.float32), ("seed", np.uint64),
           ("request", np.uint64), ("codebook", np.int32), ("row_stream", np.int32),
           ("eos_id", np.int32), ("feedback_slot", np.int32))


def _to_device(a, dtype, device):
    import torch
    arr = np.ascontiguousarray(np.asarray(a, dtype=dtype))
    if arr.dtype == np.uint64:
        arr = arr.view(np.int64)
    elif arr.dtype == np.uint16:
        arr = arr.view(np.int16)
    return torch.from_numpy(arr.copy()).to(device)


class DeviceBatch:
    """One step's inputs and outputs in device memory plus the ``ts_batch``.

    ``host`` is a workload dict (see ``workloads.make``): numpy arrays that
    are copied to ``device`` once.  ``logits`` may be replaced by any device
    tensor of the same layout (``set_logits``), e.g. to rotate step buffers.
    """

    def __init__(self, host: dict, device="cuda", feedback: bool = True,
                 advance_steps: bool = False, finish=None, history=None,
                 double_steps: bool = False):
        import torch
        self.device = torch.device(device)
        self.dtype = TS_DTYPE_BF16 if host["dtype"] == "bf16" else TS_DTYPE_F32
        self.n_rows = int(host["n_rows"])
        self.arrays = {}
        logits = np.asarray(host["logits"],
                            dtype=np.uint16 if self.dtype == TS_DTYPE_BF16 else np.float32)
        self.logits = _to_device(logits, logits.dtype, self.device)
        for name, dt in _ARRAYS:
            self.arrays[name] = _to_device(host[name], dt, self.device)
        self.step = _to_device(host["step"], np.int64, self.device)
        self.out_ids = torch.full((self.n_rows,), -2, dtype=torch.int32, device=self.device)
        self.out_eos = torch.zeros(self.n_rows, dtype=torch.uint8, device=self.device)
        self.feedback = None
        if feedback:
            self.feedback = torch.full((int(host["feedback_len"]),), -1, dtype=torch.int32,
                                       device=self.device)
        c = TsBatch()
        c.dtype = self.dtype
        c.n_rows = self.n_rows
        c.max_row_vocab = int(host.get("max_row_vocab",
                                       int(np.max(host["row_vocab"], initial=1))))
        for name, _ in _ARRAYS:
            setattr(c, name, self.arrays[name].data_ptr())
        c.step = self.step.data_ptr()
        c.n_streams = int(host["n_streams"])
        c.advance_steps = 1 if advance_steps else 0
        # double_steps: a second step array receives the advanced steps
        # (step_out); swap_steps() exchanges the two between calls
        self.step_next = None
        if double_steps:
            self.step_next = torch.empty_like(self.step)
            c.step_out = self.step_next.data_ptr()
        # finished streams: finish = {"max_steps": per-stream caps or None,
        # "pad_id": int}; stop_step starts at -1 and finish_reason at 0
        self.stop_step = self.max_steps = self.finish_reason = None
        if finish is not None:
            n_streams = int(host["n_streams"])
            self.stop_step = torch.full((n_streams,), -1, dtype=torch.int64, device=self.device)
            self.finish_reason = torch.zeros(n_streams, dtype=torch.uint8, device=self.device)
            c.stop_step = self.stop_step.data_ptr()
            c.finish_reason = self.finish_reason.data_ptr()
            if finish.get("max_steps") is not None:
                self.max_steps = _to_device(finish["max_steps"], np.int64, self.device)
                c.max_steps = self.max_steps.data_ptr()
            c.pad_id = int(finish.get("pad_id", -1))
        # repetition penalty: history = {"len": T, "codebooks": Q, "penalty":
        # per-row theta}; the ring [n_streams, T, Q] starts empty (-1)
        self.hist_ring = self.rep_penalty = None
        if history is not None:
            n_streams = int(host["n_streams"])
            self.hist_ring = torch.full((n_streams, int(history["len"]), int(history["codebooks"])),
                                        -1, dtype=torch.int32, device=self.device)
            self.rep_penalty = _to_device(history["penalty"], np.float32, self.device)
            c.hist_ring = self.hist_ring.data_ptr()
            c.hist_len = int(history["len"])
            c.hist_codebooks = int(history["codebooks"])
            c.rep_penalty = self.rep_penalty.data_ptr()
        c.out_ids = self.out_ids.data_ptr()
        c.out_eos = self.out_eos.data_ptr()
        if self.feedback is not None:
            c.feedback_buf = self.feedback.data_ptr()
            c.feedback_len = self.feedback.numel()
        else:
            c.feedback_buf = None
            c.feedback_slot = None
            c.feedback_len = 0
        self.c = c
        self.set_logits(self.logits)

    def swap_steps(self) -> None:
        """With double_steps: the array the last call wrote becomes the one the
        next call reads (host-side pointer swap; capture it between calls)."""
        if self.step_next is None:
            raise ValueError("the batch has no second step array")
        self.step, self.step_next = self.step_next, self.step
        self.c.step = self.step.data_ptr()
        self.c.step_out = self.step_next.data_ptr()

    def set_logits(self, t) -> None:
        """Point the batch at another device tensor of logits (same layout)."""
        self.logits = t
        self.c.logits = t.data_ptr()
        self.c.logits_len = t.numel()

    def ids(self) -> np.ndarray:
        return self.out_ids.cpu().numpy()

    def eos(self) -> np.ndarray:
        return self.out_eos.cpu().numpy()


class LmHead:
    """A frame's hidden states and output heads in device memory plus the
    ``ts_lm_head`` (see ``ts_lm_head_logits``).

    ``head`` is a dict of numpy arrays: ``hidden`` (bf16 bits, n_rows x dim),
    ``weights`` (bf16 bits), ``head_offsets`` (int64 per head), ``n_heads``
    and ``dim``; row r uses head r mod n_heads.  ``set_weights`` and
    ``set_hidden`` point the call at other device tensors of the same layout.
    """

    def __init__(self, head: dict, device="cuda"):
        import torch
        self.device = torch.device(device)
        self.hidden = _to_device(np.asarray(head["hidden"], np.uint16), np.uint16, self.device)
        self.weights = _to_device(np.asarray(head["weights"], np.uint16), np.uint16, self.device)
        self.head_offsets = _to_device(head["head_offsets"], np.int64, self.device)
        c = TsLmHead()
        c.head_offsets = self.head_offsets.data_ptr()
        c.dim = int(head["dim"])
        c.n_heads = int(head["n_heads"])
        self.c = c
        self.set_hidden(self.hidden)
        self.set_weights(self.weights)

    def set_hidden(self, t) -> None:
        self.hidden = t
        self.c.hidden = t.data_ptr()

    def set_weights(self, t) -> None:
        self.weights = t
        self.c.weights = t.data_ptr()
        self.c.weights_len = t.numel()


# --------------------------------------------------------------------------
# The paged key-value cache
# --------------------------------------------------------------------------
def _kv_dtype(t) -> int:
    import torch
    kinds = {torch.float32: TS_DTYPE_F32, torch.bfloat16: TS_DTYPE_BF16,
             torch.float8_e4m3fn: TS_DTYPE_E4M3}
    if t.dtype not in kinds:
        raise ValueError(f"no key-value type for {t.dtype}")
    return kinds[t.dtype]


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _vector(t, n: int, dtype, device, what: str):
    """``t``: a contiguous tensor of ``n`` entries or more of ``dtype`` on
    ``device``; its address (0 for None)."""
    if t is None:
        return None
    _need(t.dtype == dtype and t.is_contiguous() and t.numel() >= n and t.device == device, what)
    return t.data_ptr()


def _strides(t) -> list:
    """Element strides of all but the last dimension, 0 for those of one entry."""
    return [st if n > 1 else 0 for st, n in zip(t.stride()[:-1], t.shape[:-1])]


def _table_stride(t) -> int:
    """The stride of a block table's rows, which are contiguous and do not overlap
    (a row that several requests share, e.g. an expanded one, is refused); a single
    row's says nothing."""
    n, wide = t.shape
    _need((wide < 2 or t.stride(1) == 1) and (n < 2 or t.stride(0) >= wide),
          "block_table: contiguous rows of their own")
    return t.stride(0) if n > 1 else wide


class KvTables:
    """Block tables, lengths, the stack of free blocks and the slot maps of one
    cache, with a prebuilt ``ts_kv_tables_args``.

    Starts with every request empty and every block free, or from the int32
    device tensors given: ``lens`` [n], ``block_table`` [n, max_blocks] (rows
    may be strided), ``free_blocks`` and ``n_free`` [1].  ``n_new`` (int32 [n];
    None: one token each) and ``finished`` (uint8 [n], e.g. a ``DeviceBatch``'s
    ``finish_reason``) are read by every call.  With ``double`` the new lengths
    and the free count go to second arrays (``lens_out``, ``n_free_out``;
    ``swap()`` exchanges them), otherwise they are updated in place.
    """

    def __init__(self, n_requests: int, max_blocks: int, n_blocks: int, block_size: int, *,
                 max_tokens: int, lens=None, n_new=None, finished=None, block_table=None,
                 free_blocks=None, n_free=None, double: bool = False, device="cuda"):
        import torch
        i32 = torch.int32
        given = [t for t in (lens, block_table, free_blocks, n_free) if t is not None]
        dev = given[0].device if given else torch.empty(0, device=device).device

        def make(*shape, fill=0, dtype=i32):
            return torch.full(shape, fill, dtype=dtype, device=dev)
        self.lens = make(n_requests) if lens is None else lens
        self.block_table = make(n_requests, max_blocks, fill=-1) if block_table is None else block_table
        if free_blocks is None:
            free_blocks = torch.arange(n_blocks - 1, -1, -1, dtype=i32, device=dev)
        self.free_blocks = free_blocks
        self.n_free = make(1, fill=n_blocks) if n_free is None else n_free
        self.lens_out = torch.empty_like(self.lens) if double else self.lens
        self.n_free_out = torch.empty_like(self.n_free) if double else self.n_free
        self.n_new, self.finished = n_new, finished
        self.token_starts = make(n_requests + 1)
        self.slots = make(max_tokens, fill=-1, dtype=torch.int64)
        self.positions = make(max_tokens, fill=-1)
        self.requests = make(max_tokens, fill=-1)
        t = self.block_table
        _need(t.dtype == i32 and t.device == dev and tuple(t.shape) == (n_requests, max_blocks),
              "block_table: int32 [n_requests, max_blocks]")
        c = TsKvTables()
        c.n_requests, c.block_size, c.n_blocks, c.max_blocks = n_requests, block_size, n_blocks, max_blocks
        c.table_stride = _table_stride(t)
        c.block_table = t.data_ptr()
        c.free_blocks = _vector(self.free_blocks, 1 if n_blocks else 0, i32, dev, "free_blocks: int32")
        c.free_len = self.free_blocks.numel()
        c.max_tokens = max_tokens
        for name in ("token_starts", "slots", "positions", "requests"):
            setattr(c, name, getattr(self, name).data_ptr())
        self.c = c
        self._n, self._dev = n_requests, dev
        self._bind()
        self.set_requests(n_new, finished)

    def _bind(self) -> None:
        import torch
        for name, n in (("lens", self._n), ("lens_out", self._n), ("n_free", 1), ("n_free_out", 1)):
            setattr(self.c, name, _vector(getattr(self, name), n, torch.int32, self._dev,
                                          f"{name}: int32 [{n}]"))

    def set_requests(self, n_new=None, finished=None) -> None:
        """Other arrays of new tokens and ended requests for the next calls."""
        import torch
        self.n_new, self.finished = n_new, finished
        self.c.n_new = _vector(n_new, self._n, torch.int32, self._dev, "n_new: int32 [n_requests]")
        self.c.finished = _vector(finished, self._n, torch.uint8, self._dev,
                                  "finished: uint8 [n_requests]")

    def swap(self) -> None:
        """With ``double``: what the last call wrote becomes what the next one
        reads (host-side pointer swap; capture it between calls)."""
        self.lens, self.lens_out = self.lens_out, self.lens
        self.n_free, self.n_free_out = self.n_free_out, self.n_free
        self._bind()


class KvCache:
    """A paged cache with a prebuilt ``ts_kv_cache``: ``k`` and ``v`` are device
    tensors seen as [n_blocks, block_size, n_kv_heads, head_dim], in whatever
    order they lie in memory (permute a [block, head, token, dim] tensor), of
    type float32, bfloat16 or float8_e4m3fn; the 8-bit type may have float32
    scales, one per key head."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.device == v.device,
              "k and v: [n_blocks, block_size, n_kv_heads, head_dim] of one type")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "k and v: head_dim is contiguous")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        # what tokens and queries have to match: key heads, head_dim, device
        self.rows_of = (k.shape[2], k.shape[3], k.device)
        c = TsKvCache()
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.dtype = _kv_dtype(k)
        c.n_blocks, c.block_size, c.n_kv_heads, c.head_dim = k.shape
        c.k_block_stride, c.k_token_stride, c.k_head_stride = _strides(k)
        c.v_block_stride, c.v_token_stride, c.v_head_stride = _strides(v)
        c.k_scale = _vector(k_scale, k.shape[2], torch.float32, k.device, "k_scale: float32 [n_kv_heads]")
        c.v_scale = _vector(v_scale, k.shape[2], torch.float32, k.device, "v_scale: float32 [n_kv_heads]")
        self.c = c


class KvTokens:
    """New tokens' keys and values [n_rows, n_kv_heads, head_dim] (any strides
    with head_dim contiguous) and their slots, with a prebuilt ``ts_kv_tokens``.
    Token x is row x, or with ``rows`` (int32, one per slot) row ``rows[x]``."""

    def __init__(self, k, v, slots, rows=None):
        import torch
        _need(k.dim() == 3 and k.shape == v.shape and k.dtype == v.dtype and k.device == v.device,
              "k and v: [n_tokens, n_kv_heads, head_dim] of one type")
        _need(k.stride(2) == 1 and v.stride(2) == 1, "k and v: head_dim is contiguous")
        self.k, self.v, self.slots, self.rows = k, v, slots, rows
        self.rows_of = (k.shape[1], k.shape[2], k.device)
        c = TsKvTokens()
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.dtype = _kv_dtype(k)
        c.n_rows = k.shape[0]
        c.n_tokens = k.shape[0] if rows is None else rows.numel()
        c.k_token_stride, c.k_head_stride = _strides(k)
        c.v_token_stride, c.v_head_stride = _strides(v)
        c.slots = _vector(slots, c.n_tokens, torch.int64, k.device, "slots: int64 [n_tokens]")
        c.rows = _vector(rows, c.n_tokens, torch.int32, k.device, "rows: int32 [n_tokens]")
        self.c = c


class PagedQuery:
    """One query token per request [n_requests, n_heads, head_dim], its output
    and what it attends to, with a prebuilt ``ts_paged_query``.  ``scale``
    defaults to head_dim ** -0.5; ``lse`` (float32 [n_requests, n_heads]),
    ``key_mask`` (uint8 [n_requests, max_blocks * block_size or more]),
    ``window`` and ``softcap`` are optional."""

    def __init__(self, q, out, block_table, lens, *, scale=None, lse=None, key_mask=None,
                 window: int = 0, softcap: float = 0.0):
        import torch
        n, heads, dim = q.shape
        _need(q.shape == out.shape and q.dtype == out.dtype and q.device == out.device,
              "q and out: [n_requests, n_heads, head_dim] of one type")
        _need(q.stride(2) == 1 and out.stride(2) == 1, "q and out: head_dim is contiguous")
        _need(block_table.dtype == torch.int32 and block_table.dim() == 2
              and block_table.shape[0] == n and block_table.device == q.device,
              "block_table: int32 [n_requests, max_blocks]")
        self.q, self.out, self.block_table, self.lens = q, out, block_table, lens
        self.lse, self.key_mask = lse, key_mask
        self.rows_of = (dim, q.device)
        c = TsPagedQuery()
        c.q, c.out = q.data_ptr(), out.data_ptr()
        c.lse = _vector(lse, n * heads, torch.float32, q.device, "lse: float32 [n_requests, n_heads]")
        c.dtype = _kv_dtype(q)
        c.n_requests, c.n_heads, c.max_blocks = n, heads, block_table.shape[1]
        c.q_request_stride, c.q_head_stride = _strides(q)
        c.out_request_stride, c.out_head_stride = _strides(out)
        c.block_table = block_table.data_ptr()
        c.table_stride = _table_stride(block_table)
        c.lens = _vector(lens, n, torch.int32, q.device, "lens: int32 [n_requests]")
        c.key_mask = None
        if key_mask is not None:
            _need(key_mask.dtype == torch.uint8 and key_mask.dim() == 2 and key_mask.shape[0] == n
                  and key_mask.device == q.device
                  and (key_mask.shape[1] < 2 or key_mask.stride(1) == 1), "key_mask: uint8 [n_requests, tokens]")
            c.key_mask = key_mask.data_ptr()
            # a row holds this many entries; one request's stride says nothing
            c.mask_stride = key_mask.stride(0) if n > 1 else key_mask.shape[1]
        c.scale = dim ** -0.5 if scale is None else scale
        c.softcap, c.window = softcap, window
        self.c = c

    def set_lens(self, lens) -> None:
        """Another array of lengths (e.g. after ``KvTables.swap``)."""
        import torch
        self.lens = lens
        self.c.lens = _vector(lens, self.c.n_requests, torch.int32, self.q.device,
                              "lens: int32 [n_requests]")


# --------------------------------------------------------------------------
# The layer operators around it
# --------------------------------------------------------------------------
def _rows_of(t, shape, dtypes, device, what: str):
    """``t``: rows of contiguous elements [n, dim] of one of ``dtypes`` on ``device``,
    which do not overlap; its address and row stride (a single row's says nothing)."""
    _need(t.dim() == 2 and tuple(t.shape) == tuple(shape) and t.dtype in dtypes and t.device == device, what)
    n, dim = t.shape
    _need((dim < 2 or t.stride(1) == 1) and (n < 2 or t.stride(0) >= dim), f"{what}: contiguous rows of their own")
    return t.data_ptr(), t.stride(0) if n > 1 else dim


def _scales_of(t, n: int, dim: int, out, what: str):
    """The scales of 8-bit rows ``out`` of ``n`` x ``dim``, which other types do not have."""
    import torch
    _need((t is not None) == (out.dtype == torch.float8_e4m3fn), f"{what}: for 8-bit rows, and only for them")
    blocks = -(-dim // TS_SCALE_BLOCK)
    return (None, 0) if t is None else _rows_of(t, (n, blocks), (torch.float32,), out.device,
                                                f"{what}: float32 [n_rows, {blocks}]")


class RmsNorm:
    """``out`` [n, dim] = the root-mean-square norm of ``x`` (+ ``residual``, whose sum
    goes to ``residual_out``) times ``weight`` (+ ``weight_offset``), with a prebuilt
    ``ts_norm_args``.  ``x`` and ``residual`` are bfloat16 or float32, ``weight`` [dim]
    either; ``out`` is one of the two, or float8_e4m3fn with ``out_scale`` (float32
    [n, ceil(dim / 128)]).  Rows may be strided; ``residual_out`` may be ``residual`` or
    ``x``, ``out`` may be ``x``."""

    def __init__(self, x, out, weight=None, *, residual=None, residual_out=None, out_scale=None,
                 eps: float = 1e-6, weight_offset: float = 0.0):
        import torch
        real = (torch.float32, torch.bfloat16)
        _need(x.dim() == 2, "x: [n_rows, dim]")
        n, dim = x.shape
        self.x, self.out, self.weight, self.out_scale = x, out, weight, out_scale
        self.residual, self.residual_out = residual, residual_out
        c = TsNorm()
        c.x, c.x_stride = _rows_of(x, (n, dim), real, x.device, "x: bfloat16 or float32 [n_rows, dim]")
        for name, t in (("residual", residual), ("residual_out", residual_out)):
            if t is not None:
                at, stride = _rows_of(t, (n, dim), (x.dtype,), x.device, f"{name}: as x")
                setattr(c, name, at)
                setattr(c, name + "_stride", stride)
        c.out, c.out_stride = _rows_of(out, (n, dim), (*real, torch.float8_e4m3fn), x.device, "out: [n_rows, dim]")
        c.out_scale, c.out_scale_stride = _scales_of(out_scale, n, dim, out, "out_scale")
        if weight is not None:
            _need(weight.dtype in real, "weight: bfloat16 or float32")
            c.weight = _vector(weight, dim, weight.dtype, x.device, "weight: [dim]")
            c.weight_dtype = _kv_dtype(weight)
        c.dtype, c.out_dtype = _kv_dtype(x), _kv_dtype(out)
        c.n_rows, c.dim = n, dim
        c.eps, c.weight_offset = eps, weight_offset
        self.c = c


class Gate:
    """``out`` [n, dim] = activation(``gate``) * ``up``, with a prebuilt ``ts_gate_args``;
    ``activation`` is "silu", "gelu", "gelu_tanh", or "none" (``out`` = ``up``, without a
    gate).  ``up`` and ``gate`` are bfloat16 or float32, e.g. the halves of one product's
    rows; ``out`` is one of the two, or float8_e4m3fn with ``out_scale`` (float32
    [n, ceil(dim / 128)])."""

    ACTIVATIONS = {"none": TS_ACT_NONE, "silu": TS_ACT_SILU, "gelu": TS_ACT_GELU, "gelu_tanh": TS_ACT_GELU_TANH}

    def __init__(self, up, out, gate=None, *, activation: str = "silu", out_scale=None):
        import torch
        real = (torch.float32, torch.bfloat16)
        _need(activation in self.ACTIVATIONS, f"activation: one of {', '.join(self.ACTIVATIONS)}")
        _need((gate is None) == (activation == "none"), "gate: with an activation, and only with one")
        _need(up.dim() == 2, "up: [n_rows, dim]")
        n, dim = up.shape
        self.up, self.gate, self.out, self.out_scale = up, gate, out, out_scale
        c = TsGate()
        c.up, c.up_stride = _rows_of(up, (n, dim), real, up.device, "up: bfloat16 or float32 [n_rows, dim]")
        if gate is not None:
            c.gate, c.gate_stride = _rows_of(gate, (n, dim), (up.dtype,), up.device, "gate: as up")
        c.out, c.out_stride = _rows_of(out, (n, dim), (*real, torch.float8_e4m3fn), up.device, "out: [n_rows, dim]")
        c.out_scale, c.out_scale_stride = _scales_of(out_scale, n, dim, out, "out_scale")
        c.dtype, c.out_dtype, c.act = _kv_dtype(up), _kv_dtype(out), self.ACTIVATIONS[activation]
        c.n_rows, c.dim = n, dim
        self.c = c


class LinearE4m3:
    """``out`` [n, out_dim] = ``x`` [n, in_dim] times ``w`` [out_dim, in_dim] transposed,
    both float8_e4m3fn with float32 scales, ``x_scale`` for each row's 128 elements [n,
    ceil(in_dim / 128)] and ``w_scale`` for each 128 x 128 of the weights; ``out`` is
    bfloat16 or float32.  With a prebuilt ``ts_linear_args``."""

    def __init__(self, x, x_scale, w, w_scale, out):
        import torch
        e4m3, f32 = (torch.float8_e4m3fn,), (torch.float32,)
        _need(x.dim() == 2 and w.dim() == 2, "x: [n_rows, in_dim], w: [out_dim, in_dim]")
        n, k = x.shape
        m = w.shape[0]
        blocks = -(-k // TS_SCALE_BLOCK)
        self.x, self.x_scale, self.w, self.w_scale, self.out = x, x_scale, w, w_scale, out
        c = TsLinear()
        c.x, c.x_stride = _rows_of(x, (n, k), e4m3, x.device, "x: float8_e4m3fn [n_rows, in_dim]")
        c.x_scale, c.x_scale_stride = _rows_of(x_scale, (n, blocks), f32, x.device, f"x_scale: float32 [n_rows, {blocks}]")
        c.w, c.w_stride = _rows_of(w, (m, k), e4m3, x.device, "w: float8_e4m3fn [out_dim, in_dim]")
        c.w_scale, c.w_scale_stride = _rows_of(w_scale, (-(-m // TS_SCALE_BLOCK), blocks), f32, x.device,
                                               f"w_scale: float32 [ceil(out_dim / 128), {blocks}]")
        c.out, c.out_stride = _rows_of(out, (n, m), (torch.bfloat16, torch.float32), x.device,
                                       "out: bfloat16 or float32 [n_rows, out_dim]")
        c.out_dtype, c.n_rows, c.in_dim, c.out_dim = _kv_dtype(out), n, k, m
        self.c = c


class Rotary:
    """Rotary positions of the heads ``x`` [n_rows, n_heads, head_dim] (bfloat16 or float32,
    any strides with head_dim contiguous) to ``out`` (which may be ``x``), with a prebuilt
    ``ts_rotary_args``.  Token t is row t, or with ``rows`` (int32) row ``rows[t]``;
    ``positions`` (int32) below 0 skip it.  ``freqs`` (float64 [rotary_dim / 2] on the
    device, see ``ts_rotary_frequencies``) gives the width that is turned; ``interleaved``
    pairs neighbours instead of halves."""

    def __init__(self, x, out, positions, freqs, *, rows=None, interleaved: bool = False,
                 amplitude: float = 1.0):
        import torch
        _need(x.dim() == 3 and x.shape == out.shape and x.dtype == out.dtype and x.device == out.device,
              "x and out: [n_rows, n_heads, head_dim] of one type")
        _need(x.dtype in (torch.float32, torch.bfloat16), "x and out: bfloat16 or float32")
        _need(x.shape[2] < 2 or (x.stride(2) == 1 and out.stride(2) == 1), "x and out: head_dim is contiguous")
        _need(freqs.dim() == 1 and 0 < 2 * freqs.numel() <= x.shape[2], "freqs: [rotary_dim / 2], at most head_dim / 2")
        self.x, self.out, self.positions, self.freqs, self.rows = x, out, positions, freqs, rows
        self.rows_of = (x.shape[2], x.device)
        c = TsRotary()
        c.x, c.out, c.dtype = x.data_ptr(), out.data_ptr(), _kv_dtype(x)
        c.n_rows, c.n_heads, c.head_dim = x.shape
        c.n_tokens = x.shape[0] if rows is None else rows.numel()
        c.rotary_dim, c.interleaved, c.amplitude = 2 * freqs.numel(), int(interleaved), amplitude
        c.x_token_stride, c.x_head_stride = _strides(x)
        c.out_token_stride, c.out_head_stride = _strides(out)
        c.positions = _vector(positions, c.n_tokens, torch.int32, x.device, "positions: int32 [n_tokens]")
        c.rows = _vector(rows, c.n_tokens, torch.int32, x.device, "rows: int32 [n_tokens]")
        c.freqs = _vector(freqs, freqs.numel(), torch.float64, x.device, "freqs: float64 [rotary_dim / 2]")
        self.c = c
