"""Python binding of the KDA CUDA library (libkda.so, C ABI in include/kda.h).

Argument marshalling only: every function checks its tensors' shapes and dtypes against the layouts the
header states, passes their device pointers and the current CUDA stream to the C entry point of the same
name, and raises KdaError on a non-OK status.  There is no CPU fallback: if the library is not built,
every call fails.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import _build

__all__ = [
    "KdaError", "load", "lib_path", "KDA_OK", "KDA_DEV_SLOT_OOB", "KDA_DEV_SEQ_OOB", "KDA_DEV_TIMEOUT",
    "KDA_DEV_ACCEPT_OOB", "KDA_DEV_POS_OOB", "KDA_DEV_PAGE_OOB", "KDA_DEV_TOKEN_OOB", "KDA_DEV_PROB_OOB", "kda_status_string", "kda_version", "kda_state_bytes_per_head", "kda_state_copy",
    "kda_decode_step", "kda_replay_bytes", "kda_verify", "kda_verify_replay", "kda_prefill_varlen",
    "kda_prefill_workspace_size", "kda_prefill_segmented", "kda_segmented_workspace_size",
    "kda_segment_fragments", "kda_fragment_scan", "kda_segment_outputs", "kda_prefill_segmented_noalloc",
    "kda_prefill_records", "kda_prefill_chain", "kda_cfbi_cache_bytes_per_head", "kda_cfbi_prefill",
    "kda_cfbi_prefill_chunked_workspace_size", "kda_cfbi_prefill_chunked",
    "kda_cfbi_decode", "kda_backward_workspace_size", "kda_prefill_backward", "kda_fused_decode",
    "kda_kcp_fragments", "kda_kcp_scan", "kda_kcp_outputs", "kda_check_slot_ids", "kda_set_debug_checks",
    "kda_qk_norm_rope", "kda_qk_norm_rope_backward", "kda_qk_norm_rope_backward_workspace_size", "kda_kv_write",
    "kda_kv_read", "kda_paged_attention", "kda_paged_attention_workspace_size", "kda_prefill_attention",
    "kda_prefill_attention_backward", "kda_prefill_attention_backward_workspace_size", "kda_verify_accept",
    "kda_debug_checks", "kda_set_test_fault", "KDA_TEST_FAULT_NONE", "KDA_TEST_FAULT_STALL_RECORD_INPUTS", "KDA_TEST_FAULT_STALL_CACHE_COPIES", "KDA_TEST_FAULT_STALL_PROMPT_COPIES",
    "CFBI_CHUNK", "CFBI_ROW_FLOATS", "EXPORTED_SYMBOLS",
]

KDA_OK = 0
KDA_TEST_FAULT_NONE, KDA_TEST_FAULT_STALL_RECORD_INPUTS, KDA_TEST_FAULT_STALL_CACHE_COPIES = 0, 1, 2
KDA_TEST_FAULT_STALL_PROMPT_COPIES = 3
KDA_DEV_SLOT_OOB, KDA_DEV_SEQ_OOB, KDA_DEV_TIMEOUT, KDA_DEV_ACCEPT_OOB = 1, 2, 4, 8
KDA_DEV_POS_OOB, KDA_DEV_PAGE_OOB, KDA_DEV_TOKEN_OOB, KDA_DEV_PROB_OOB = 16, 32, 64, 128
F32, BF16 = 0, 1
CFBI_CHUNK, CFBI_ROW_FLOATS = 16, 420  # KDA_CFBI_CHUNK, KDA_CFBI_ROW_FLOATS

# every function include/kda.h declares
EXPORTED_SYMBOLS = (
    "kda_status_string", "kda_version", "kda_state_bytes_per_head", "kda_prefill_args_bytes", "kda_state_copy",
    "kda_decode_step", "kda_replay_bytes", "kda_verify", "kda_verify_replay", "kda_prefill_varlen",
    "kda_prefill_workspace_size", "kda_prefill_segmented", "kda_segmented_workspace_size",
    "kda_segment_fragments", "kda_fragment_scan", "kda_segment_outputs", "kda_prefill_segmented_noalloc",
    "kda_prefill_records", "kda_prefill_chain", "kda_cfbi_cache_bytes_per_head", "kda_cfbi_prefill",
    "kda_cfbi_prefill_chunked_workspace_size", "kda_cfbi_prefill_chunked",
    "kda_cfbi_decode", "kda_backward_args_bytes", "kda_backward_workspace_size", "kda_prefill_backward",
    "kda_fused_decode_args_bytes", "kda_fused_decode", "kda_kcp_fragments", "kda_kcp_scan", "kda_kcp_outputs",
    "kda_check_slot_ids", "kda_set_debug_checks", "kda_debug_checks", "kda_set_test_fault",
    "kda_qk_norm_rope_args_bytes", "kda_qk_norm_rope", "kda_qk_norm_rope_backward_workspace_size",
    "kda_qk_norm_rope_backward", "kda_kv_cache_bytes", "kda_kv_write", "kda_kv_read",
    "kda_paged_attention_args_bytes", "kda_paged_attention_workspace_size", "kda_paged_attention",
    "kda_prefill_attention_args_bytes", "kda_prefill_attention", "kda_prefill_attention_grads_bytes",
    "kda_prefill_attention_backward_workspace_size", "kda_prefill_attention_backward", "kda_verify_accept_args_bytes",
    "kda_verify_accept",
)


class KdaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {kda_status_string(code)} ({code})")
        self.code = code


class PrefillArgs(ctypes.Structure):
    """Mirror of kda_prefill_args."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("g", ctypes.c_void_p),
        ("beta", ctypes.c_void_p), ("in_dtype", ctypes.c_int), ("T", ctypes.c_int64), ("H", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("N", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p),
        ("max_seqlen", ctypes.c_int32), ("pool", ctypes.c_void_p), ("num_slots", ctypes.c_int32),
        ("slot_ids", ctypes.c_void_p), ("init_zero", ctypes.c_int), ("out", ctypes.c_void_p),
        ("out_dtype", ctypes.c_int), ("extra_pool", ctypes.c_void_p), ("num_extra_slots", ctypes.c_int32),
        ("extra_slot_ids", ctypes.c_void_p), ("snapshot_every_chunks", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("dev_status", ctypes.c_void_p),
    ]


class BackwardArgs(ctypes.Structure):
    """Mirror of kda_backward_args."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("g", ctypes.c_void_p),
        ("beta", ctypes.c_void_p), ("in_dtype", ctypes.c_int), ("T", ctypes.c_int64), ("H", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("N", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p),
        ("max_seqlen", ctypes.c_int32), ("pool", ctypes.c_void_p), ("num_slots", ctypes.c_int32),
        ("slot_ids", ctypes.c_void_p), ("init_zero", ctypes.c_int), ("d_out", ctypes.c_void_p),
        ("d_final", ctypes.c_void_p), ("dq", ctypes.c_void_p), ("dk_out", ctypes.c_void_p),
        ("dv_out", ctypes.c_void_p), ("dg", ctypes.c_void_p), ("dbeta", ctypes.c_void_p),
        ("d_init", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("dev_status", ctypes.c_void_p),
    ]


class FusedDecodeArgs(ctypes.Structure):
    """Mirror of kda_fused_decode_args."""
    _fields_ = [
        ("xq", ctypes.c_void_p), ("xk", ctypes.c_void_p), ("xv", ctypes.c_void_p), ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p), ("z", ctypes.c_void_p), ("in_dtype", ctypes.c_int), ("B", ctypes.c_int),
        ("H", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("pool", ctypes.c_void_p),
        ("num_slots", ctypes.c_int32), ("slot_ids", ctypes.c_void_p), ("conv_state", ctypes.c_void_p),
        ("conv_w", ctypes.c_void_p), ("norm_w", ctypes.c_void_p), ("norm_eps", ctypes.c_float),
        ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int), ("dev_status", ctypes.c_void_p),
    ]


class QkNormRopeArgs(ctypes.Structure):
    """Mirror of kda_qk_norm_rope_args."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("in_dtype", ctypes.c_int), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("num_positions", ctypes.c_int32), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
        ("eps", ctypes.c_float), ("T", ctypes.c_int64), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("d", ctypes.c_int), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64), ("out_dtype", ctypes.c_int),
        ("dev_status", ctypes.c_void_p),
    ]


class KvCache(ctypes.Structure):
    """Mirror of kda_kv_cache."""
    _fields_ = [
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p), ("type", ctypes.c_int), ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int),
    ]


class PagedAttentionArgs(ctypes.Structure):
    """Mirror of kda_paged_attention_args."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_dtype", ctypes.c_int), ("B", ctypes.c_int), ("W", ctypes.c_int),
        ("Hq", ctypes.c_int), ("cache", KvCache), ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int32),
        ("seq_lens", ctypes.c_void_p), ("scale", ctypes.c_float), ("softcap", ctypes.c_float),
        ("window", ctypes.c_int32), ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("dev_status", ctypes.c_void_p),
    ]


class PrefillAttentionArgs(ctypes.Structure):
    """Mirror of kda_prefill_attention_args."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("in_dtype", ctypes.c_int), ("T", ctypes.c_int64),
        ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("N", ctypes.c_int),
        ("cu_seqlens", ctypes.c_void_p), ("max_seqlen", ctypes.c_int32), ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float), ("window", ctypes.c_int32), ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
        ("out_dtype", ctypes.c_int), ("lse", ctypes.c_void_p), ("dev_status", ctypes.c_void_p),
    ]


class PrefillAttentionGrads(ctypes.Structure):
    """Mirror of kda_prefill_attention_grads."""
    _fields_ = [
        ("d_out", ctypes.c_void_p), ("d_out_stride", ctypes.c_int64), ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p),
        ("dv", ctypes.c_void_p), ("dq_stride", ctypes.c_int64), ("dk_stride", ctypes.c_int64),
        ("dv_stride", ctypes.c_int64), ("grad_dtype", ctypes.c_int), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class VerifyAcceptArgs(ctypes.Structure):
    """Mirror of kda_verify_accept_args."""
    _fields_ = [
        ("target_probs", ctypes.c_void_p), ("draft_probs", ctypes.c_void_p), ("dtype", ctypes.c_int), ("B", ctypes.c_int),
        ("W", ctypes.c_int), ("V", ctypes.c_int), ("draft_tokens", ctypes.c_void_p), ("num_drafts", ctypes.c_void_p),
        ("uniform", ctypes.c_void_p), ("accepted", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
        ("dev_status", ctypes.c_void_p),
    ]


def _packer(mirror):
    """struct.Struct.pack for a mirror's fields in their native layout, a nested struct's fields in its place."""
    codes = {ctypes.c_void_p: "P", ctypes.c_int: "i", ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_size_t: "N",
             ctypes.c_float: "f"}

    def fields(m):
        return "".join(codes[t] if t in codes else fields(t) for _, t in m._fields_) + "0P"  # structs end on a pointer's
    packed = struct.Struct("@" + fields(mirror))
    if packed.size != ctypes.sizeof(mirror):
        raise RuntimeError(f"{mirror.__name__}: the packed layout differs from the mirror's")
    return packed.pack


_pack_norm, _pack_cache, _pack_attention = map(_packer, (QkNormRopeArgs, KvCache, PagedAttentionArgs))
_pack_prompt, _pack_grads, _pack_accept = map(_packer, (PrefillAttentionArgs, PrefillAttentionGrads, VerifyAcceptArgs))
_packed = {}
_lib = None


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """Loads libkda.so; raises if it is not built (no fallback path exists)."""
    global _lib, _packed
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        if not build_if_missing:
            raise RuntimeError(f"KDA CUDA library not built ({_build.LIB}); run __graft_entry__.build()")
        _build.build()
    lib = ctypes.CDLL(_build.LIB)
    vp, i32, i64, sz, c_int = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    st = ctypes.c_char_p  # a packed argument struct
    sig = {
        "kda_status_string": (ctypes.c_char_p, [c_int]),
        "kda_version": (c_int, []),
        "kda_state_bytes_per_head": (sz, [c_int, c_int]),
        "kda_prefill_args_bytes": (sz, []),
        "kda_state_copy": (c_int, [vp, i32, vp, vp, i32, vp, i32, i64, vp, vp]),
        "kda_decode_step": (c_int, [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, vp, i32, vp, vp, c_int,
                                    vp, vp]),
        "kda_replay_bytes": (sz, [c_int, c_int, c_int, c_int, c_int, c_int]),
        "kda_verify": (c_int, [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, vp, i32, vp, vp, c_int,
                               vp, sz, vp, vp, vp]),
        "kda_verify_replay": (c_int, [vp, i32, vp, c_int, c_int, c_int, c_int, c_int, c_int, vp, sz, vp, vp, vp]),
        "kda_prefill_varlen": (c_int, [ctypes.POINTER(PrefillArgs), vp]),
        "kda_prefill_workspace_size": (sz, [ctypes.POINTER(PrefillArgs)]),
        "kda_prefill_segmented": (c_int, [ctypes.POINTER(PrefillArgs), i32, vp]),
        "kda_segmented_workspace_size": (sz, [ctypes.POINTER(PrefillArgs), i32]),
        "kda_segment_fragments": (c_int, [ctypes.POINTER(PrefillArgs), i32, vp]),
        "kda_fragment_scan": (c_int, [ctypes.POINTER(PrefillArgs), i32, vp]),
        "kda_segment_outputs": (c_int, [ctypes.POINTER(PrefillArgs), i32, vp]),
        "kda_prefill_segmented_noalloc": (c_int, [ctypes.POINTER(PrefillArgs), i32, vp]),
        "kda_prefill_records": (c_int, [ctypes.POINTER(PrefillArgs), vp]),
        "kda_prefill_chain": (c_int, [ctypes.POINTER(PrefillArgs), vp]),
        "kda_cfbi_cache_bytes_per_head": (sz, [c_int, c_int]),
        "kda_cfbi_prefill": (c_int, [vp, vp, vp, vp, vp, vp, i32, i64, i32, c_int, c_int, c_int, c_int, vp, vp, vp,
                                     i32, vp, vp, c_int, vp, vp]),
        "kda_cfbi_prefill_chunked_workspace_size": (sz, [i64, i32, c_int, c_int, c_int]),
        "kda_cfbi_prefill_chunked": (c_int, [vp, vp, vp, vp, vp, vp, i32, i64, i32, c_int, c_int, c_int, c_int, vp,
                                             vp, vp, i32, vp, vp, c_int, vp, sz, vp, vp]),
        "kda_cfbi_decode": (c_int, [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, vp, vp, vp, i32, vp, vp,
                                    c_int, vp, vp]),
        "kda_backward_args_bytes": (sz, []),
        "kda_backward_workspace_size": (sz, [ctypes.POINTER(BackwardArgs)]),
        "kda_prefill_backward": (c_int, [ctypes.POINTER(BackwardArgs), vp]),
        "kda_fused_decode_args_bytes": (sz, []),
        "kda_fused_decode": (c_int, [ctypes.POINTER(FusedDecodeArgs), vp]),
        "kda_kcp_fragments": (c_int, [ctypes.POINTER(PrefillArgs), i32, vp, vp]),
        "kda_kcp_scan": (c_int, [vp, i32, c_int, c_int, c_int, vp, vp, vp, vp]),
        "kda_kcp_outputs": (c_int, [ctypes.POINTER(PrefillArgs), i32, vp, vp]),
        "kda_check_slot_ids": (c_int, [vp, i32, vp, i32]),
        "kda_set_debug_checks": (None, [c_int]),
        "kda_debug_checks": (c_int, []),
        "kda_set_test_fault": (c_int, [c_int]),
        "kda_qk_norm_rope_args_bytes": (sz, []),
        "kda_qk_norm_rope": (c_int, [ctypes.POINTER(QkNormRopeArgs), vp]),
        "kda_qk_norm_rope_backward_workspace_size": (sz, [i64, c_int, c_int, c_int]),
        "kda_qk_norm_rope_backward": (c_int, [ctypes.POINTER(QkNormRopeArgs), vp, vp, c_int, vp, vp, vp, sz, vp]),
        "kda_kv_cache_bytes": (sz, []),
        "kda_kv_write": (c_int, [vp, vp, i64, i64, c_int, i64, vp, ctypes.POINTER(KvCache), vp, vp]),
        "kda_kv_read": (c_int, [ctypes.POINTER(KvCache), vp, i64, vp, vp, c_int, vp, vp]),
        "kda_paged_attention_args_bytes": (sz, []),
        "kda_paged_attention_workspace_size": (sz, [c_int, c_int, c_int, c_int, c_int]),
        "kda_paged_attention": (c_int, [ctypes.POINTER(PagedAttentionArgs), vp]),
        "kda_prefill_attention_args_bytes": (sz, []),
        "kda_prefill_attention": (c_int, [ctypes.POINTER(PrefillAttentionArgs), vp]),
        "kda_prefill_attention_grads_bytes": (sz, []),
        "kda_prefill_attention_backward_workspace_size": (sz, [i64, c_int, c_int, c_int, c_int]),
        "kda_prefill_attention_backward": (c_int, [ctypes.POINTER(PrefillAttentionArgs),
                                                   ctypes.POINTER(PrefillAttentionGrads), vp]),
        "kda_verify_accept_args_bytes": (sz, []),
        "kda_verify_accept": (c_int, [ctypes.POINTER(VerifyAcceptArgs), vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.kda_prefill_args_bytes() != ctypes.sizeof(PrefillArgs):
        raise RuntimeError("kda_prefill_args layout mismatch between include/kda.h and the binding")
    if lib.kda_backward_args_bytes() != ctypes.sizeof(BackwardArgs):
        raise RuntimeError("kda_backward_args layout mismatch between include/kda.h and the binding")
    if lib.kda_fused_decode_args_bytes() != ctypes.sizeof(FusedDecodeArgs):
        raise RuntimeError("kda_fused_decode_args layout mismatch between include/kda.h and the binding")
    for name, mirror in (("kda_qk_norm_rope_args", QkNormRopeArgs), ("kda_kv_cache", KvCache),
                         ("kda_paged_attention_args", PagedAttentionArgs),
                         ("kda_prefill_attention_args", PrefillAttentionArgs),
                         ("kda_prefill_attention_grads", PrefillAttentionGrads),
                         ("kda_verify_accept_args", VerifyAcceptArgs)):
        if getattr(lib, name + "_bytes")() != ctypes.sizeof(mirror):
            raise RuntimeError(f"{name} layout mismatch between include/kda.h and the binding")
    # The attention calls' argument structs go over as packed bytes (their mirrors cost a microsecond to fill, more than
    # the rest of such a call's marshalling); function objects of their own, since the pointer type differs.
    packed = {}
    for name, args in (("kda_qk_norm_rope", [st, vp]), ("kda_qk_norm_rope_backward", [st, vp, vp, c_int, vp, vp, vp, sz, vp]),
                       ("kda_kv_write", [vp, vp, i64, i64, c_int, i64, vp, st, vp, vp]),
                       ("kda_kv_read", [st, vp, i64, vp, vp, c_int, vp, vp]), ("kda_paged_attention", [st, vp]),
                       ("kda_prefill_attention", [st, vp]), ("kda_prefill_attention_backward", [st, st, vp]),
                       ("kda_verify_accept", [st, vp])):
        packed[name] = lib[name]
        packed[name].restype, packed[name].argtypes = c_int, args
    _packed = packed  # whole: another thread's call takes a table that is there for a loaded library
    _lib = lib
    return lib


# ---------------------------------------------------------------- marshalling helpers

def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_DTYPE_CODES = {torch.float32: F32, torch.bfloat16: BF16}


def _dt(t: torch.Tensor) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


# torch.cuda.current_stream() builds a Stream object (3 us on the host); this returns its handle alone
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("expected contiguous CUDA tensors")


# Shapes and dtypes, checked on the host before the device check and before any call into the library.
# The C ABI takes bare pointers and the kernels trust the extents they are given, so a tensor of the wrong
# shape or dtype would be read or written out of bounds on the device instead of raising here.  A shape
# entry of None accepts any extent.

_FP = (torch.float32,)
_IN = (torch.float32, torch.bfloat16)
_I32 = (torch.int32,)


def _need(name, t, shape, dtypes):
    if t is None or (t.shape == shape and t.dtype in dtypes):  # the common case first: None entries fail it
        return
    if t.dim() != len(shape) or any(s is not None and t.shape[i] != s for i, s in enumerate(shape)):
        want = ", ".join("*" if s is None else str(s) for s in shape)
        raise ValueError(f"{name}: expected shape [{want}], got {list(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected dtype {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")


def _need_status(t):
    if t is not None and (t.dtype != torch.int32 or t.numel() < 2):
        raise ValueError(f"dev_status: expected an int32 tensor of at least 2 elements, got {t.dtype} "
                         f"x {t.numel()}")


def _rank(name, t, n):
    if t.dim() != n:
        raise ValueError(f"{name}: expected {n} dimensions, got shape {list(t.shape)}")
    return tuple(t.shape)


def _need_tokens(q, k, v, g, beta, lead):
    """q, k, g [*lead, H, dk]; v [*lead, H, dv] in q's dtype (fp32 or bf16); g fp32; beta [*lead, H] fp32.
    Returns (H, dk, dv)."""
    n = len(lead)
    H, dk = _rank("q", q, n + 2)[n:]
    _need("q", q, (*lead, H, dk), _IN)
    _need("k", k, (*lead, H, dk), (q.dtype,))
    _need("v", v, (*lead, H, None), (q.dtype,))
    dv = v.shape[-1]
    _need("g", g, (*lead, H, dk), _FP)
    _need("beta", beta, (*lead, H), _FP)
    return H, dk, dv


def _need_prefill(q, k, v, g, beta, cu_seqlens, pool, slot_ids, out, extra_pool=None, extra_slot_ids=None):
    T = _rank("q", q, 3)[0]
    H, dk, dv = _need_tokens(q, k, v, g, beta, (T,))
    _need("cu_seqlens", cu_seqlens, (None,), _I32)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens: expected N + 1 >= 1 offsets")
    N = cu_seqlens.numel() - 1
    _need("pool", pool, (None, H, dk, dv), _FP)
    _need("slot_ids", slot_ids, (N,), _I32)
    _need("out", out, (T, H, dv), _IN)
    if (extra_pool is None) != (extra_slot_ids is None):
        raise ValueError("extra_pool and extra_slot_ids go together")
    _need("extra_pool", extra_pool, (None, H, dk, dv), _FP)
    _need("extra_slot_ids", extra_slot_ids, (N, 2), _I32)
    return T, N, H, dk, dv


def _need_cfbi_cache(pool, cache, counts):
    S, H = pool.shape[:2]
    _need("cache", cache, (S, H, CFBI_CHUNK, CFBI_ROW_FLOATS), _FP)
    _need("counts", counts, (S, H), _I32)


def _ok(fn: str, code: int):
    if code != KDA_OK:
        raise KdaError(fn, code)


# ---------------------------------------------------------------- entry points

def kda_status_string(code: int) -> str:
    return load().kda_status_string(code).decode()


def kda_version() -> int:
    return load().kda_version()


def kda_check_slot_ids(ids, other_ids=None) -> int:
    """Host-side slot-id contract check on int32 host arrays (numpy or CPU tensors): KDA_OK when the ids are
    distinct and none is among other_ids, else the error code (include/kda.h)."""
    import numpy as np
    a = np.ascontiguousarray(np.asarray(ids), dtype=np.int32)
    b = None if other_ids is None else np.ascontiguousarray(np.asarray(other_ids), dtype=np.int32)
    return load().kda_check_slot_ids(a.ctypes.data if a.size else None, a.size,
                                     None if b is None or not b.size else b.ctypes.data, 0 if b is None else b.size)


def kda_set_debug_checks(on: bool):
    """Switch the library's debug mode (host-side slot-id checks before every call that takes slot ids)."""
    load().kda_set_debug_checks(1 if on else 0)


def kda_set_test_fault(fault: int):
    """Test hook for the kernels' bounded waits (include/kda.h): KDA_TEST_FAULT_STALL_RECORD_INPUTS makes
    kda_prefill_records' first input wait give up and flag KDA_DEV_TIMEOUT; KDA_TEST_FAULT_NONE restores."""
    _ok("kda_set_test_fault", load().kda_set_test_fault(int(fault)))


def kda_debug_checks() -> bool:
    return bool(load().kda_debug_checks())


def kda_state_bytes_per_head(dk: int, dv: int) -> int:
    return load().kda_state_bytes_per_head(dk, dv)


def kda_state_copy(src_pool, src_slots, dst_pool, dst_slots, dev_status=None, stream=None):
    """dst_pool[dst_slots[i]] = src_pool[src_slots[i]] (pools [slots, H, dk, dv] fp32)."""
    head = _rank("src_pool", src_pool, 4)[1:]
    _need("src_pool", src_pool, (None, *head), _FP)
    _need("dst_pool", dst_pool, (None, *head), _FP)
    _need("src_slots", src_slots, (None,), _I32)
    _need("dst_slots", dst_slots, (src_slots.numel(),), _I32)
    _need_status(dev_status)
    _check(src_pool, src_slots, dst_pool, dst_slots, dev_status)
    n = src_slots.numel()
    elems = src_pool[0].numel() if src_pool.shape[0] else dst_pool[0].numel()
    _ok("kda_state_copy", load().kda_state_copy(_p(src_pool), src_pool.shape[0], _p(src_slots), _p(dst_pool),
                                                dst_pool.shape[0], _p(dst_slots), n, elems, _p(dev_status),
                                                _stream(stream)))


def kda_decode_step(q, k, v, g, beta, pool, slot_ids, out, dev_status=None, stream=None):
    """One token per request; q, k, g [B, H, dk]; v, out [B, H, dv]; beta [B, H]; pool updated in place."""
    B = _rank("q", q, 3)[0]
    H, dk, dv = _need_tokens(q, k, v, g, beta, (B,))
    _need("pool", pool, (None, H, dk, dv), _FP)
    _need("slot_ids", slot_ids, (B,), _I32)
    _need("out", out, (B, H, dv), _IN)
    _need_status(dev_status)
    _check(q, k, v, g, beta, pool, slot_ids, out, dev_status)
    B, H, dk = q.shape
    dv = v.shape[-1]
    _ok("kda_decode_step", load().kda_decode_step(_p(q), _p(k), _p(v), _p(g), _p(beta), B, H, dk, dv, _dt(q),
                                                  _p(pool), pool.shape[0], _p(slot_ids), _p(out), _dt(out),
                                                  _p(dev_status), _stream(stream)))


def kda_cfbi_cache_bytes_per_head(dk: int = 128, dv: int = 128) -> int:
    return load().kda_cfbi_cache_bytes_per_head(dk, dv)


def kda_cfbi_prefill(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, cache, counts, slot_ids, out, dev_status=None,
                     stream=None):
    """CF-BI prefill over packed sequences: q, k, g [T, H, 128]; v, out [T, H, 128]; beta [T, H];
    cu_seqlens int32 [N + 1]; pool [S, H, 128, 128]; cache [S, H, 16, 420] fp32; counts [S, H] int32."""
    _need_prefill(q, k, v, g, beta, cu_seqlens, pool, slot_ids, out)
    _need_cfbi_cache(pool, cache, counts)
    _need_status(dev_status)
    _check(q, k, v, g, beta, cu_seqlens, pool, cache, counts, slot_ids, out, dev_status)
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    _ok("kda_cfbi_prefill", load().kda_cfbi_prefill(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), N, T,
                                                    int(max_seqlen), H, dk, dv, _dt(q), _p(pool), _p(cache),
                                                    _p(counts), pool.shape[0], _p(slot_ids), _p(out), _dt(out),
                                                    _p(dev_status), _stream(stream)))


def kda_cfbi_prefill_chunked_workspace_size(T: int, N: int, H: int, dk: int = 128, dv: int = 128) -> int:
    return load().kda_cfbi_prefill_chunked_workspace_size(int(T), int(N), int(H), int(dk), int(dv))


def kda_cfbi_prefill_chunked(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, cache, counts, slot_ids, out,
                             workspace, dev_status=None, stream=None):
    """kda_cfbi_prefill with the chunks worked on in parallel (same arguments and the same bits); workspace is
    a uint8 device tensor of at least kda_cfbi_prefill_chunked_workspace_size(T, N, H) bytes."""
    _need_prefill(q, k, v, g, beta, cu_seqlens, pool, slot_ids, out)
    _need_cfbi_cache(pool, cache, counts)
    _need_status(dev_status)
    _check(q, k, v, g, beta, cu_seqlens, pool, cache, counts, slot_ids, out, dev_status, workspace)
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    _ok("kda_cfbi_prefill_chunked",
        load().kda_cfbi_prefill_chunked(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), N, T, int(max_seqlen),
                                        H, dk, dv, _dt(q), _p(pool), _p(cache), _p(counts), pool.shape[0],
                                        _p(slot_ids), _p(out), _dt(out), _p(workspace),
                                        workspace.numel() * workspace.element_size(), _p(dev_status),
                                        _stream(stream)))


def kda_cfbi_decode(q, k, v, g, beta, pool, cache, counts, slot_ids, out, dev_status=None, stream=None):
    """CF-BI decode, one token per request: q, k, g [B, H, 128]; v, out [B, H, 128]; beta [B, H]."""
    B = _rank("q", q, 3)[0]
    H, dk, dv = _need_tokens(q, k, v, g, beta, (B,))
    _need("pool", pool, (None, H, dk, dv), _FP)
    _need("slot_ids", slot_ids, (B,), _I32)
    _need("out", out, (B, H, dv), _IN)
    _need_cfbi_cache(pool, cache, counts)
    _need_status(dev_status)
    _check(q, k, v, g, beta, pool, cache, counts, slot_ids, out, dev_status)
    B, H, dk = q.shape
    dv = v.shape[-1]
    _ok("kda_cfbi_decode", load().kda_cfbi_decode(_p(q), _p(k), _p(v), _p(g), _p(beta), B, H, dk, dv, _dt(q),
                                                  _p(pool), _p(cache), _p(counts), pool.shape[0], _p(slot_ids),
                                                  _p(out), _dt(out), _p(dev_status), _stream(stream)))


def kda_replay_bytes(B: int, W: int, H: int, dk: int, dv: int, in_dtype: int) -> int:
    return load().kda_replay_bytes(B, W, H, dk, dv, in_dtype)


def kda_verify(q, k, v, g, beta, pool, slot_ids, out, replay, snapshot_out=None, dev_status=None, stream=None):
    """Draft window: q, k, g [B, W, H, dk]; v, out [B, W, H, dv]; beta [B, W, H]; replay: uint8 record buffer."""
    B, W = _rank("q", q, 4)[:2]
    H, dk, dv = _need_tokens(q, k, v, g, beta, (B, W))
    _need("pool", pool, (None, H, dk, dv), _FP)
    _need("slot_ids", slot_ids, (B,), _I32)
    _need("out", out, (B, W, H, dv), _IN)
    _need("snapshot_out", snapshot_out, (B, W, H, dk, dv), _FP)
    _need_status(dev_status)
    _check(q, k, v, g, beta, pool, slot_ids, out, replay, snapshot_out, dev_status)
    B, W, H, dk = q.shape
    dv = v.shape[-1]
    _ok("kda_verify", load().kda_verify(_p(q), _p(k), _p(v), _p(g), _p(beta), B, W, H, dk, dv, _dt(q), _p(pool),
                                        pool.shape[0], _p(slot_ids), _p(out), _dt(out), _p(replay),
                                        replay.numel() * replay.element_size(), _p(snapshot_out), _p(dev_status),
                                        _stream(stream)))


def kda_verify_replay(pool, slot_ids, replay, accepted_len, W, H, dk, dv, in_dtype, dev_status=None, stream=None):
    """Commits tokens 1..accepted_len[b] of each window into pool[slot_ids[b]]."""
    _need("pool", pool, (None, H, dk, dv), _FP)
    _need("slot_ids", slot_ids, (None,), _I32)
    _need("accepted_len", accepted_len, (slot_ids.numel(),), _I32)
    _need_status(dev_status)
    _check(pool, slot_ids, replay, accepted_len, dev_status)
    B = slot_ids.numel()
    _ok("kda_verify_replay", load().kda_verify_replay(_p(pool), pool.shape[0], _p(slot_ids), B, W, H, dk, dv,
                                                      in_dtype, _p(replay), replay.numel() * replay.element_size(),
                                                      _p(accepted_len), _p(dev_status), _stream(stream)))


def _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero=False,
                    extra_pool=None, extra_slot_ids=None, snapshot_every_chunks=0, workspace=None, dev_status=None):
    _need_prefill(q, k, v, g, beta, cu_seqlens, pool, slot_ids, out, extra_pool, extra_slot_ids)
    _need_status(dev_status)
    _check(q, k, v, g, beta, cu_seqlens, pool, slot_ids, out, extra_pool, extra_slot_ids, workspace, dev_status)
    T, H, dk = q.shape
    a = PrefillArgs()
    a.q, a.k, a.v, a.g, a.beta = (t.data_ptr() for t in (q, k, v, g, beta))
    a.in_dtype = _dt(q)
    a.T, a.H, a.dk, a.dv = T, H, dk, v.shape[-1]
    a.N = cu_seqlens.numel() - 1
    a.cu_seqlens = cu_seqlens.data_ptr()
    a.max_seqlen = int(max_seqlen)
    a.pool, a.num_slots, a.slot_ids = pool.data_ptr(), pool.shape[0], slot_ids.data_ptr()
    a.init_zero = int(bool(init_zero))
    a.out, a.out_dtype = out.data_ptr(), _dt(out)
    if extra_pool is not None:
        a.extra_pool, a.num_extra_slots = extra_pool.data_ptr(), extra_pool.shape[0]
        a.extra_slot_ids = extra_slot_ids.data_ptr()
        a.snapshot_every_chunks = int(snapshot_every_chunks)
    if workspace is not None:
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if dev_status is not None:
        a.dev_status = dev_status.data_ptr()
    return a


def kda_prefill_varlen(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero=False,
                       extra_pool=None, extra_slot_ids=None, snapshot_every_chunks=0, workspace=None,
                       dev_status=None, stream=None):
    """Packed prefill: q, k, g [T, H, dk]; v, out [T, H, dv]; beta [T, H]; cu_seqlens int32 [N+1]."""
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero, extra_pool,
                        extra_slot_ids, snapshot_every_chunks, workspace, dev_status)
    _ok("kda_prefill_varlen", load().kda_prefill_varlen(ctypes.byref(a), _stream(stream)))


def kda_prefill_records(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero=False,
                        extra_pool=None, extra_slot_ids=None, snapshot_every_chunks=0, workspace=None,
                        dev_status=None, stream=None):
    """Phase 1 of the tensor-core prefill: per-chunk operand records into `workspace`."""
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero, extra_pool,
                        extra_slot_ids, snapshot_every_chunks, workspace, dev_status)
    _ok("kda_prefill_records", load().kda_prefill_records(ctypes.byref(a), _stream(stream)))


def kda_prefill_chain(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero=False,
                      extra_pool=None, extra_slot_ids=None, snapshot_every_chunks=0, workspace=None,
                      dev_status=None, stream=None):
    """Phase 2 of the tensor-core prefill: the state carry over the chunks, from the records."""
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero, extra_pool,
                        extra_slot_ids, snapshot_every_chunks, workspace, dev_status)
    _ok("kda_prefill_chain", load().kda_prefill_chain(ctypes.byref(a), _stream(stream)))


def kda_prefill_workspace_size(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, **kw) -> int:
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, **kw)
    return load().kda_prefill_workspace_size(ctypes.byref(a))


def kda_segmented_workspace_size(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, segment_len,
                                 **kw) -> int:
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, **kw)
    return load().kda_segmented_workspace_size(ctypes.byref(a), int(segment_len))


def _segmented(fn, q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, segment_len, workspace,
               init_zero=False, extra_pool=None, extra_slot_ids=None, snapshot_every_chunks=0, dev_status=None,
               stream=None):
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero, extra_pool,
                        extra_slot_ids, snapshot_every_chunks, workspace, dev_status)
    _ok(fn, getattr(load(), fn)(ctypes.byref(a), int(segment_len), _stream(stream)))


def kda_prefill_segmented(*args, **kw):
    """Segmented (KCP) prefill; same arguments as kda_prefill_varlen plus segment_len and workspace."""
    _segmented("kda_prefill_segmented", *args, **kw)


def kda_segment_fragments(*args, **kw):
    _segmented("kda_segment_fragments", *args, **kw)


def kda_fragment_scan(*args, **kw):
    _segmented("kda_fragment_scan", *args, **kw)


def kda_segment_outputs(*args, **kw):
    _segmented("kda_segment_outputs", *args, **kw)


def kda_prefill_segmented_noalloc(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, segment_len,
                                  init_zero=False, extra_pool=None, extra_slot_ids=None, snapshot_every_chunks=0,
                                  dev_status=None, stream=None):
    """kda_prefill_segmented without a caller workspace: for callers that cannot allocate device memory,
    the scratch comes from a fixed 32 MiB array inside the library (see include/kda.h)."""
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, init_zero, extra_pool,
                        extra_slot_ids, snapshot_every_chunks, None, dev_status)
    _ok("kda_prefill_segmented_noalloc",
        load().kda_prefill_segmented_noalloc(ctypes.byref(a), int(segment_len), _stream(stream)))


def _backward_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, d_out, dq, dk, dv, dg, dbeta, pool=None,
                     slot_ids=None, d_final=None, d_init=None, workspace=None, dev_status=None):
    T = _rank("q", q, 3)[0]
    H, d_k, d_v = _need_tokens(q, k, v, g, beta, (T,))
    _need("cu_seqlens", cu_seqlens, (None,), _I32)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens: expected N + 1 >= 1 offsets")
    N = cu_seqlens.numel() - 1
    if (pool is None) != (slot_ids is None):
        raise ValueError("pool and slot_ids go together (both None: zero initial states)")
    _need("pool", pool, (None, H, d_k, d_v), _FP)
    _need("slot_ids", slot_ids, (N,), _I32)
    _need("d_out", d_out, (T, H, d_v), (q.dtype,))
    for name, t, w in (("dq", dq, d_k), ("dk", dk, d_k), ("dg", dg, d_k), ("dv", dv, d_v)):
        _need(name, t, (T, H, w), _FP)
    _need("dbeta", dbeta, (T, H), _FP)
    _need("d_final", d_final, (N, H, d_k, d_v), _FP)
    _need("d_init", d_init, (N, H, d_k, d_v), _FP)
    _need_status(dev_status)
    _check(q, k, v, g, beta, cu_seqlens, d_out, dq, dk, dv, dg, dbeta, pool, slot_ids, d_final, d_init, workspace,
           dev_status)
    T, H, dkk = q.shape
    a = BackwardArgs()
    a.q, a.k, a.v, a.g, a.beta = (t.data_ptr() for t in (q, k, v, g, beta))
    a.in_dtype = _dt(q)
    a.T, a.H, a.dk, a.dv = T, H, dkk, v.shape[-1]
    a.N = cu_seqlens.numel() - 1
    a.cu_seqlens = cu_seqlens.data_ptr()
    a.max_seqlen = int(max_seqlen)
    if pool is None:
        a.init_zero = 1
    else:
        a.pool, a.num_slots, a.slot_ids = pool.data_ptr(), pool.shape[0], slot_ids.data_ptr()
    a.d_out = d_out.data_ptr()
    a.dq, a.dk_out, a.dv_out, a.dg, a.dbeta = (t.data_ptr() for t in (dq, dk, dv, dg, dbeta))
    if d_final is not None:
        a.d_final = d_final.data_ptr()
    if d_init is not None:
        a.d_init = d_init.data_ptr()
    if workspace is not None:
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if dev_status is not None:
        a.dev_status = dev_status.data_ptr()
    return a


def kda_backward_workspace_size(T: int, N: int, H: int, dk: int = 128, dv: int = 128) -> int:
    a = BackwardArgs()
    a.T, a.N, a.H, a.dk, a.dv = T, N, H, dk, dv
    return load().kda_backward_workspace_size(ctypes.byref(a))


def kda_prefill_backward(q, k, v, g, beta, cu_seqlens, max_seqlen, d_out, dq, dk, dv, dg, dbeta, workspace,
                         pool=None, slot_ids=None, d_final=None, d_init=None, dev_status=None, stream=None):
    """Gradients of sum <d_out, o> + <d_final, S_T> through the packed prefill of (q, k, v, g, beta).

    q, k, g, dq, dk, dg [T, H, 128]; v, d_out, dv [T, H, 128]; beta, dbeta [T, H]; cu_seqlens int32 [N + 1];
    initial states pool[slot_ids] (or zero when pool is None); d_final, d_init [N, H, 128, 128] fp32 or None;
    workspace: >= kda_backward_workspace_size(T, N, H) bytes.  Outputs are fp32.
    """
    a = _backward_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, d_out, dq, dk, dv, dg, dbeta, pool, slot_ids,
                         d_final, d_init, workspace, dev_status)
    _ok("kda_prefill_backward", load().kda_prefill_backward(ctypes.byref(a), _stream(stream)))


def kda_fused_decode(xq, xk, xv, a, b, z, pool, slot_ids, conv_state, conv_w, norm_w, out, norm_eps=1e-5,
                     dev_status=None, stream=None):
    """One decode token per request through the short convolution, the KDA step and the gated output norm.

    xq, xk, xv, z, out [B, H, 128]; a [B, H, 128]; b [B, H]; pool [S, H, 128, 128];
    conv_state [S, H, 3, 3, 128] fp32 (advanced in place); conv_w [3, H, 128, 4]; norm_w [128].
    """
    B, H, d = _rank("xq", xq, 3)
    _need("xq", xq, (B, H, d), _IN)
    for name, t in (("xk", xk), ("xv", xv), ("z", z)):
        _need(name, t, (B, H, d), (xq.dtype,))
    _need("a", a, (B, H, d), _FP)
    _need("b", b, (B, H), _FP)
    _need("pool", pool, (None, H, d, d), _FP)
    _need("slot_ids", slot_ids, (B,), _I32)
    _need("conv_state", conv_state, (pool.shape[0], H, 3, 3, d), _FP)
    _need("conv_w", conv_w, (3, H, d, 4), _FP)
    _need("norm_w", norm_w, (d,), _FP)
    _need("out", out, (B, H, d), _IN)
    _need_status(dev_status)
    _check(xq, xk, xv, a, b, z, pool, slot_ids, conv_state, conv_w, norm_w, out, dev_status)
    B, H, d = xq.shape
    f = FusedDecodeArgs()
    f.xq, f.xk, f.xv, f.a, f.b, f.z = (t.data_ptr() for t in (xq, xk, xv, a, b, z))
    f.in_dtype = _dt(xq)
    f.B, f.H, f.dk, f.dv = B, H, d, d
    f.pool, f.num_slots, f.slot_ids = pool.data_ptr(), pool.shape[0], slot_ids.data_ptr()
    f.conv_state, f.conv_w, f.norm_w = conv_state.data_ptr(), conv_w.data_ptr(), norm_w.data_ptr()
    f.norm_eps = float(norm_eps)
    f.out, f.out_dtype = out.data_ptr(), _dt(out)
    if dev_status is not None:
        f.dev_status = dev_status.data_ptr()
    _ok("kda_fused_decode", load().kda_fused_decode(ctypes.byref(f), _stream(stream)))


def kda_kcp_fragments(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, segment_len, workspace, frag_out,
                      dev_status=None, stream=None):
    """Fragments (S~ | M) of every segment of the shard's sequences, the last included, into frag_out
    [N, P, H, dk, dv + dk]; run kda_prefill_records on the same workspace first (tensor-core path)."""
    _, N, H, dk, dv = _need_prefill(q, k, v, g, beta, cu_seqlens, pool, slot_ids, out)
    _need("frag_out", frag_out, (N, None, H, dk, dv + dk), _FP)
    _check(frag_out)
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, workspace=workspace,
                        dev_status=dev_status)
    _ok("kda_kcp_fragments", load().kda_kcp_fragments(ctypes.byref(a), int(segment_len), _p(frag_out),
                                                      _stream(stream)))


def kda_kcp_scan(frags, s0, entries, dev_status=None, stream=None):
    """entries[0] = s0, entries[p + 1] = M_p entries[p] + S~_p over gathered fragments [P, H, dk, dv + dk]."""
    P, H, dk, w = _rank("frags", frags, 4)
    dv = w - dk
    _need("frags", frags, (P, H, dk, dv + dk), _FP)
    _need("s0", s0, (H, dk, dv), _FP)
    _need("entries", entries, (P, H, dk, dv), _FP)
    _need_status(dev_status)
    _check(frags, s0, entries, dev_status)
    P, H, dk, w = frags.shape
    _ok("kda_kcp_scan", load().kda_kcp_scan(_p(frags), P, H, dk, w - dk, _p(s0), _p(entries), _p(dev_status),
                                            _stream(stream)))


def kda_kcp_outputs(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, segment_len, workspace, entries,
                    dev_status=None, stream=None):
    """Outputs and final states of the shard from its entry states [N, P, H, dk, dv]."""
    _, N, H, dk, dv = _need_prefill(q, k, v, g, beta, cu_seqlens, pool, slot_ids, out)
    _need("entries", entries, (N, None, H, dk, dv), _FP)
    _check(entries)
    a = _prefill_struct(q, k, v, g, beta, cu_seqlens, max_seqlen, pool, slot_ids, out, workspace=workspace,
                        dev_status=dev_status)
    _ok("kda_kcp_outputs", load().kda_kcp_outputs(ctypes.byref(a), int(segment_len), _p(entries), _stream(stream)))


# ---------------------------------------------------------------- softmax-attention layers

_I64 = (torch.int64,)
_CACHE_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}  # KDA_CACHE_BF16, KDA_CACHE_E4M3


def _row_stride(name, t):
    """Elements between the tokens of t [T, H, d], whose heads and channels must be contiguous: a tensor of its own
    or a column block of a fused projection's output."""
    T, H, d = t.shape
    st, sh, sc = t.stride()
    if not t.is_cuda or (sc != 1 and d > 1) or (sh != d and H > 1):
        raise ValueError(f"{name}: expected contiguous CUDA tensors, or heads and channels contiguous within a token")
    return st if T > 1 else H * d


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _call(name, *args):
    if not _packed:
        load()
    code = _packed[name](*args)
    if code != KDA_OK:
        raise KdaError(name, code)


# The checks of these calls are written twice: one expression that the usual call passes (a call of one token spends
# most of its time here), and behind it the checks one by one, which name what is wrong.

def _qk_norm_checks(q, k, q_weight, k_weight, q_out, k_out, out_names, cos, sin, positions, dev_status, grads,
                    weight_grads):
    T, Hq, d = _rank("q", q, 3)
    _need("q", q, q.shape, _IN)
    _need("k", k, (T, k.shape[1] if k.dim() == 3 else None, d), (q.dtype,))
    _need("q_weight", q_weight, (d,), _FP)
    _need("k_weight", k_weight, (d,), _FP)
    _need(out_names[0], q_out, q.shape, _IN)
    _need(out_names[1], k_out, k.shape, (q_out.dtype,))
    if cos is not None or sin is not None or positions is not None:
        if cos is None or sin is None or positions is None:
            raise ValueError("cos, sin and positions go together (all None: no rotation)")
        half = _rank("cos", cos, 2)[1]
        _need("cos", cos, cos.shape, _FP)
        _need("sin", sin, cos.shape, _FP)
        _need("positions", positions, (T,), _I32)
        if 2 * half > d or half % 8:
            raise ValueError(f"cos: expected angles of a multiple of 8 channel pairs within d = {d}, got {half}")
    if grads:
        _need("d_q_out", grads[0], q.shape, _IN)
        _need("d_k_out", grads[1], k.shape, (grads[0].dtype,))
        _need("dq_weight", weight_grads[0], (d,), _FP)
        _need("dk_weight", weight_grads[1], (d,), _FP)
    _need_status(dev_status)
    _check(q_weight, k_weight, dev_status, cos, sin, positions, *grads, *weight_grads)


def _qk_norm_args(q, k, q_weight, k_weight, q_out, k_out, out_names, cos, sin, positions, eps, interleaved, dev_status,
                  grads=(), weight_grads=()):
    shape, k_shape, dtype, out_dtype, f32 = q.shape, k.shape, q.dtype, q_out.dtype, torch.float32
    w_shape, in_code, out_code = shape[2:], _DTYPE_CODES.get(dtype), _DTYPE_CODES.get(out_dtype)
    n = rot = 0
    usual = (len(shape) == 3 and len(k_shape) == 3 and k_shape[0] == shape[0] and k_shape[2] == shape[2]
             and k.dtype is dtype and in_code is not None and out_code is not None and k_out.dtype is out_dtype
             and q_out.shape == shape and k_out.shape == k_shape and q_weight.shape == w_shape
             and k_weight.shape == w_shape and q_weight.dtype is f32 and k_weight.dtype is f32 and q_weight.is_cuda
             and k_weight.is_cuda and q_weight.is_contiguous() and k_weight.is_contiguous() and dev_status is None)
    if grads and usual:
        (d_q, d_k), (w_q, w_k) = grads, weight_grads
        usual = (d_q.shape == shape and d_k.shape == k_shape and d_q.dtype in _DTYPE_CODES and d_k.dtype is d_q.dtype
                 and w_q.shape == w_shape and w_k.shape == w_shape and w_q.dtype is f32 and w_k.dtype is f32
                 and d_q.is_cuda and d_k.is_cuda and w_q.is_cuda and w_k.is_cuda and d_q.is_contiguous()
                 and d_k.is_contiguous() and w_q.is_contiguous() and w_k.is_contiguous())
    if cos is not None and usual and sin is not None and positions is not None:
        c_shape = cos.shape
        usual = (len(c_shape) == 2 and c_shape[1] % 8 == 0 and 2 * c_shape[1] <= shape[2] and sin.shape == c_shape
                 and cos.dtype is f32 and sin.dtype is f32 and positions.shape == shape[:1]
                 and positions.dtype is torch.int32 and cos.is_cuda and sin.is_cuda and positions.is_cuda
                 and cos.is_contiguous() and sin.is_contiguous() and positions.is_contiguous())
    elif cos is not None or sin is not None or positions is not None:
        usual = False
    if not usual:
        _qk_norm_checks(q, k, q_weight, k_weight, q_out, k_out, out_names, cos, sin, positions, dev_status, grads,
                        weight_grads)
    if cos is not None:
        n, rot = cos.shape
        rot *= 2
    T, Hq, d = shape
    Hkv = k_shape[1]
    return _pack_norm(q.data_ptr(), k.data_ptr(), _row_stride("q", q), _row_stride("k", k), in_code,
                      q_weight.data_ptr(), k_weight.data_ptr(), _ptr(cos), _ptr(sin), _ptr(positions), n, rot,
                      bool(interleaved), eps, T, Hq, Hkv, d, q_out.data_ptr(), k_out.data_ptr(),
                      _row_stride(out_names[0], q_out), _row_stride(out_names[1], k_out), out_code, _ptr(dev_status))


def kda_qk_norm_rope(q, k, q_weight, k_weight, q_out, k_out, cos=None, sin=None, positions=None, eps=1e-6,
                     interleaved=False, dev_status=None, stream=None):
    """RMS norm of every query and key head and their position rotation, in one pass.

    q, q_out [T, Hq, d]; k, k_out [T, Hkv, d], each with any distance between tokens (column blocks of a fused
    projection's output, say), q_out and k_out may be q and k; weights [d] fp32; cos, sin [positions, rot / 2] fp32
    and positions int32 [T], or all None for no rotation.
    """
    a = _qk_norm_args(q, k, q_weight, k_weight, q_out, k_out, ("q_out", "k_out"), cos, sin, positions, eps, interleaved,
                      dev_status)
    _call("kda_qk_norm_rope", a, _stream(stream))


def kda_qk_norm_rope_backward_workspace_size(T: int, Hq: int, Hkv: int, d: int) -> int:
    return load().kda_qk_norm_rope_backward_workspace_size(T, Hq, Hkv, d)


def kda_qk_norm_rope_backward(d_q_out, d_k_out, q, k, q_weight, k_weight, dq, dk, dq_weight, dk_weight, workspace,
                              cos=None, sin=None, positions=None, eps=1e-6, interleaved=False, dev_status=None,
                              stream=None):
    """Gradients of sum <d_q_out, q_out> + <d_k_out, k_out> through kda_qk_norm_rope of (q, k, weights).

    d_q_out, dq [T, Hq, d]; d_k_out, dk [T, Hkv, d]; dq_weight, dk_weight [d] fp32 (overwritten); workspace: at least
    kda_qk_norm_rope_backward_workspace_size(T, Hq, Hkv, d) bytes.
    """
    a = _qk_norm_args(q, k, q_weight, k_weight, dq, dk, ("dq", "dk"), cos, sin, positions, eps, interleaved, dev_status,
                      (d_q_out, d_k_out), (dq_weight, dk_weight))
    _check(workspace)
    _call("kda_qk_norm_rope_backward", a, d_q_out.data_ptr(), d_k_out.data_ptr(), _dt(d_q_out), dq_weight.data_ptr(),
          dk_weight.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))


def _kv_cache(k_pages, v_pages, k_scales, v_scales):
    """The fields of kda_kv_cache."""
    shape, dtype = k_pages.shape, k_pages.dtype
    kind = _CACHE_TYPES.get(dtype)
    if not (kind is not None and v_pages.shape == shape and v_pages.dtype is dtype and shape[2] > 0 and shape[2] % 16 == 0
            and k_pages.is_cuda and v_pages.is_cuda and k_pages.is_contiguous() and v_pages.is_contiguous()
            and (k_scales is None and v_scales is None if kind == 0 else
                 k_scales is not None and v_scales is not None and k_scales.shape == shape[:3] == v_scales.shape
                 and k_scales.dtype is torch.float32 and v_scales.dtype is torch.float32 and k_scales.is_cuda
                 and v_scales.is_cuda and k_scales.is_contiguous() and v_scales.is_contiguous())):
        if kind is None:
            raise TypeError(f"k_pages: expected dtype torch.bfloat16 or torch.float8_e4m3fn, got {dtype}")
        _need("v_pages", v_pages, shape, (dtype,))
        if shape[2] <= 0 or shape[2] % 16:
            raise ValueError(f"k_pages: expected pages of a positive multiple of 16 tokens, got {shape[2]}")
        if kind == 1:
            if k_scales is None or v_scales is None:
                raise ValueError("k_scales and v_scales: an e4m3 cache needs both")
            _need("k_scales", k_scales, shape[:3], _FP)
            _need("v_scales", v_scales, shape[:3], _FP)
        elif k_scales is not None or v_scales is not None:
            raise ValueError("k_scales and v_scales: a bfloat16 cache has none")
        _check(k_pages, v_pages, k_scales, v_scales)
    pages, Hkv, page_size, d = shape
    return (k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales), _ptr(v_scales), kind, pages, page_size, Hkv, d)


def kda_kv_write(k, v, k_pages, v_pages, slots, k_scales=None, v_scales=None, dev_status=None, stream=None):
    """Token t of k, v [T, Hkv, d] goes to cache slot slots[t] = page * page_size + offset (int64, distinct; negative:
    skipped).  k_pages, v_pages [pages, Hkv, page_size, d] bfloat16, or float8_e4m3fn with k_scales, v_scales
    [pages, Hkv, page_size] fp32: each row quantised with a power-of-two scale of its own."""
    shape, page_shape = k.shape, k_pages.shape
    code = _DTYPE_CODES.get(k.dtype)
    if not (len(shape) == 3 and len(page_shape) == 4 and shape[1] == page_shape[1] and shape[2] == page_shape[3]
            and code is not None and v.shape == shape and v.dtype is k.dtype and slots.shape == shape[:1]
            and slots.dtype is torch.int64 and slots.is_cuda and slots.is_contiguous() and dev_status is None):
        T = _rank("k", k, 3)[0]
        _, Hkv, _, d = _rank("k_pages", k_pages, 4)
        _need("k", k, (T, Hkv, d), _IN)
        _need("v", v, k.shape, (k.dtype,))
        _need("slots", slots, (T,), _I64)
        _need_status(dev_status)
        _kv_cache(k_pages, v_pages, k_scales, v_scales)
        _check(slots, dev_status)
    c = _pack_cache(*_kv_cache(k_pages, v_pages, k_scales, v_scales))
    _call("kda_kv_write", k.data_ptr(), v.data_ptr(), _row_stride("k", k), _row_stride("v", v), code, shape[0],
          slots.data_ptr(), c, _ptr(dev_status), _stream(stream))


def kda_kv_read(k_pages, v_pages, slots, k_out, v_out, k_scales=None, v_scales=None, dev_status=None, stream=None):
    """Token t of k_out, v_out [T, Hkv, d] receives cache slot slots[t] (int64; negative: a zero row)."""
    shape, page_shape = k_out.shape, k_pages.shape
    code = _DTYPE_CODES.get(k_out.dtype)
    if not (len(shape) == 3 and len(page_shape) == 4 and shape[1] == page_shape[1] and shape[2] == page_shape[3]
            and code is not None and v_out.shape == shape and v_out.dtype is k_out.dtype and slots.shape == shape[:1]
            and slots.dtype is torch.int64 and slots.is_cuda and k_out.is_cuda and v_out.is_cuda
            and slots.is_contiguous() and k_out.is_contiguous() and v_out.is_contiguous() and dev_status is None):
        _, Hkv, _, d = _rank("k_pages", k_pages, 4)
        T = _rank("slots", slots, 1)[0]
        _need("slots", slots, (T,), _I64)
        _need("k_out", k_out, (T, Hkv, d), _IN)
        _need("v_out", v_out, k_out.shape, (k_out.dtype,))
        _need_status(dev_status)
        _kv_cache(k_pages, v_pages, k_scales, v_scales)
        _check(slots, k_out, v_out, dev_status)
    c = _pack_cache(*_kv_cache(k_pages, v_pages, k_scales, v_scales))
    _call("kda_kv_read", c, slots.data_ptr(), shape[0], k_out.data_ptr(), v_out.data_ptr(), code, _ptr(dev_status),
          _stream(stream))


def kda_paged_attention_workspace_size(B: int, W: int, Hq: int, Hkv: int, d: int) -> int:
    return load().kda_paged_attention_workspace_size(B, W, Hq, Hkv, d)


def kda_paged_attention(q, k_pages, v_pages, block_table, seq_lens, out, workspace, k_scales=None, v_scales=None,
                        scale=None, softcap=0.0, window=0, lse=None, dev_status=None, stream=None):
    """Attention of the W newest tokens of each request over its cached tokens (the new ones written first).

    q, out [B, W, Hq, d]; pages and scales as kda_kv_write; block_table int32 [B, max_pages]; seq_lens int32 [B], the
    tokens in the cache; scale: 1 / sqrt(d) unless given; softcap > 0: scores softcap * tanh(x / softcap);
    window > 0: a query sees that many positions, its own included; lse [B, W, Hq] fp32 or None; workspace: at least
    kda_paged_attention_workspace_size(B, W, Hq, Hkv, d) bytes.
    """
    shape, page_shape, table_shape = q.shape, k_pages.shape, block_table.shape
    code, out_code, i32 = _DTYPE_CODES.get(q.dtype), _DTYPE_CODES.get(out.dtype), torch.int32
    if not (len(shape) == 4 and len(page_shape) == 4 and shape[3] == page_shape[3] and page_shape[1] > 0
            and shape[2] % page_shape[1] == 0 and code is not None and out_code is not None and out.shape == shape
            and len(table_shape) == 2 and table_shape[0] == shape[0] and block_table.dtype is i32
            and seq_lens.shape == shape[:1] and seq_lens.dtype is i32 and q.is_cuda and out.is_cuda
            and block_table.is_cuda and seq_lens.is_cuda and workspace.is_cuda and q.is_contiguous()
            and out.is_contiguous() and block_table.is_contiguous() and seq_lens.is_contiguous()
            and workspace.is_contiguous() and dev_status is None
            and (lse is None or (lse.shape == shape[:3] and lse.dtype is torch.float32 and lse.is_cuda
                                 and lse.is_contiguous()))):
        B, W, Hq, d = _rank("q", q, 4)
        pages, Hkv, page_size, dc = _rank("k_pages", k_pages, 4)
        _need("q", q, q.shape, _IN)
        if dc != d:
            _need("k_pages", k_pages, (pages, Hkv, page_size, d), (k_pages.dtype,))
        _need("block_table", block_table, (B, _rank("block_table", block_table, 2)[1]), _I32)
        _need("seq_lens", seq_lens, (B,), _I32)
        _need("out", out, q.shape, _IN)
        _need("lse", lse, q.shape[:3], _FP)
        if Hkv == 0 or Hq % Hkv:
            raise ValueError(f"q: expected a multiple of the cache's {Hkv} heads, got {Hq}")
        _need_status(dev_status)
        _kv_cache(k_pages, v_pages, k_scales, v_scales)
        _check(q, block_table, seq_lens, out, lse, workspace, dev_status)
    c = _kv_cache(k_pages, v_pages, k_scales, v_scales)
    B, W, Hq, d = shape
    a = _pack_attention(q.data_ptr(), code, B, W, Hq, *c, block_table.data_ptr(), table_shape[1], seq_lens.data_ptr(),
                        d ** -0.5 if scale is None else scale, softcap, window, out.data_ptr(), out_code, _ptr(lse),
                        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _ptr(dev_status))
    _call("kda_paged_attention", a, _stream(stream))


# ---------------------------------------------------------------- prompts of the attention layers, and accepted drafts

def _same_device(*named):
    """Every tensor on the current device: the launches go there."""
    here = torch.cuda.current_device()
    for name, t in named:
        if t is not None and t.get_device() != here:
            raise ValueError(f"{name}: expected a tensor on the current device cuda:{here}, got {t.device}")


def _prompt_checks(q, k, v, cu_seqlens, out, lse, dev_status, grads):
    T, Hq, d = _rank("q", q, 3)
    _need("q", q, q.shape, _IN)
    Hkv = _rank("k", k, 3)[1]
    _need("k", k, (T, Hkv, d), (q.dtype,))
    _need("v", v, (T, Hkv, d), (q.dtype,))
    if Hkv == 0 or Hq % Hkv:
        raise ValueError(f"q: expected a multiple of the keys' {Hkv} heads, got {Hq}")
    _need("cu_seqlens", cu_seqlens, (None,), _I32)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens: expected N + 1 >= 1 offsets")
    _need("out", out, q.shape, _IN)
    _need("lse", lse, (T, Hq), _FP)
    if grads:
        d_out, dq, dk, dv = grads
        _need("d_out", d_out, q.shape, (q.dtype,))
        _need("dq", dq, q.shape, _IN)
        _need("dk", dk, k.shape, (dq.dtype,))
        _need("dv", dv, k.shape, (dq.dtype,))
    _need_status(dev_status)
    _check(cu_seqlens, lse, dev_status)


def _prompt_args(q, k, v, cu_seqlens, max_seqlen, out, scale, softcap, window, lse, dev_status, grads=()):
    shape, k_shape, dtype, lens = q.shape, k.shape, q.dtype, cu_seqlens.shape
    code, out_code = _DTYPE_CODES.get(dtype), _DTYPE_CODES.get(out.dtype)
    usual = (len(shape) == 3 and len(k_shape) == 3 and k_shape[0] == shape[0] and k_shape[2] == shape[2] and k_shape[1] > 0
             and shape[1] % k_shape[1] == 0 and v.shape == k_shape and k.dtype is dtype and v.dtype is dtype
             and code is not None and out_code is not None and out.shape == shape and len(lens) == 1 and lens[0] > 0
             and cu_seqlens.dtype is torch.int32 and cu_seqlens.is_cuda and cu_seqlens.is_contiguous() and dev_status is None
             and (lse is None or (lse.shape == shape[:2] and lse.dtype is torch.float32 and lse.is_cuda
                                  and lse.is_contiguous())))
    if grads and usual:
        d_out, dq, dk, dv = grads
        usual = (d_out.shape == shape and d_out.dtype is dtype and dq.shape == shape and dk.shape == k_shape
                 and dv.shape == k_shape and dq.dtype in _DTYPE_CODES and dk.dtype is dq.dtype and dv.dtype is dq.dtype)
    if not usual:
        _prompt_checks(q, k, v, cu_seqlens, out, lse, dev_status, grads)
    T, Hq, d = shape
    strides = _row_stride("q", q), _row_stride("k", k), _row_stride("v", v)
    out_stride = _row_stride("out", out)
    _same_device(("q", q), ("k", k), ("v", v), ("cu_seqlens", cu_seqlens), ("out", out), ("lse", lse),
                 ("dev_status", dev_status))
    return _pack_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides, code, T, Hq, k_shape[1], d, lens[0] - 1,
                        cu_seqlens.data_ptr(), max_seqlen, d ** -0.5 if scale is None else scale, softcap, window,
                        out.data_ptr(), out_stride, out_code, _ptr(lse), _ptr(dev_status))


def kda_prefill_attention(q, k, v, cu_seqlens, max_seqlen, out, scale=None, softcap=0.0, window=0, lse=None,
                          dev_status=None, stream=None):
    """Causal attention of whole prompts, packed one behind another.

    q, out [T, Hq, d]; k, v [T, Hkv, d], each with any distance between tokens (column blocks of a fused projection's
    output, say); cu_seqlens int32 [N + 1]; max_seqlen: at least the longest sequence; scale: 1 / sqrt(d) unless given;
    softcap > 0: scores softcap * tanh(x / softcap); window > 0: a query sees that many positions, its own included;
    lse [T, Hq] fp32 or None (the gradient needs it).
    """
    a = _prompt_args(q, k, v, cu_seqlens, max_seqlen, out, scale, softcap, window, lse, dev_status)
    _call("kda_prefill_attention", a, _stream(stream))


def kda_prefill_attention_backward_workspace_size(T: int, N: int, Hq: int, Hkv: int, d: int) -> int:
    return load().kda_prefill_attention_backward_workspace_size(T, N, Hq, Hkv, d)


def kda_prefill_attention_backward(d_out, q, k, v, out, lse, cu_seqlens, max_seqlen, dq, dk, dv, workspace, scale=None,
                                   softcap=0.0, window=0, dev_status=None, stream=None):
    """Gradients of sum <d_out, out> through kda_prefill_attention of (q, k, v), which returned out and lse.

    d_out, dq [T, Hq, d]; dk, dv [T, Hkv, d] (overwritten; column blocks of one buffer are allowed); workspace: at least
    kda_prefill_attention_backward_workspace_size(T, N, Hq, Hkv, d) bytes; the rest as in the forward call.
    """
    if lse is None:
        raise ValueError("lse: the gradient needs the forward's")
    a = _prompt_args(q, k, v, cu_seqlens, max_seqlen, out, scale, softcap, window, lse, dev_status, (d_out, dq, dk, dv))
    strides = _row_stride("d_out", d_out), _row_stride("dq", dq), _row_stride("dk", dk), _row_stride("dv", dv)
    _check(workspace)
    _same_device(("d_out", d_out), ("dq", dq), ("dk", dk), ("dv", dv), ("workspace", workspace))
    g = _pack_grads(d_out.data_ptr(), strides[0], dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *strides[1:], _dt(dq),
                    workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _call("kda_prefill_attention_backward", a, g, _stream(stream))


def kda_verify_accept(target_probs, draft_tokens, uniform, accepted, tokens, draft_probs=None, num_drafts=None,
                      dev_status=None, stream=None):
    """Which drafts of each request's window the target accepts, and the token drawn behind them.

    target_probs [B, W, V] fp32 or bf16; draft_tokens int32 [B, W - 1] (window tokens 1 .. W - 1); uniform [B, W] fp32 in
    [0, 1): one number per draft, the last for the draw; accepted int32 [B]: window tokens to commit, as
    kda_verify_replay takes it (accepted drafts + 1); tokens int32 [B, W]: accepted drafts, the drawn token, then -1;
    draft_probs [B, W - 1, V] like target_probs, or None for drafts that were certain; num_drafts int32 [B] or None.
    """
    shape, code, i32 = target_probs.shape, _DTYPE_CODES.get(target_probs.dtype), torch.int32
    if not (len(shape) == 3 and shape[1] > 0 and shape[2] > 0 and code is not None
            and draft_tokens.shape == (shape[0], shape[1] - 1) and draft_tokens.dtype is i32 and uniform.shape == shape[:2]
            and uniform.dtype is torch.float32 and accepted.shape == shape[:1] and accepted.dtype is i32
            and tokens.shape == shape[:2] and tokens.dtype is i32 and num_drafts is None and dev_status is None
            and (draft_probs is None or (draft_probs.shape == (shape[0], shape[1] - 1, shape[2])
                                         and draft_probs.dtype is target_probs.dtype))):
        B, W, V = _rank("target_probs", target_probs, 3)
        _need("target_probs", target_probs, target_probs.shape, _IN)
        if W == 0 or V == 0:
            raise ValueError(f"target_probs: expected a window and a vocabulary of at least one, got {list(shape)}")
        _need("draft_tokens", draft_tokens, (B, W - 1), _I32)
        _need("uniform", uniform, (B, W), _FP)
        _need("accepted", accepted, (B,), _I32)
        _need("tokens", tokens, (B, W), _I32)
        _need("draft_probs", draft_probs, (B, W - 1, V), (target_probs.dtype,))
        _need("num_drafts", num_drafts, (B,), _I32)
        _need_status(dev_status)
    _check(target_probs, draft_tokens, uniform, accepted, tokens, draft_probs, num_drafts, dev_status)
    _same_device(("target_probs", target_probs), ("draft_tokens", draft_tokens), ("uniform", uniform), ("accepted", accepted),
                 ("tokens", tokens), ("draft_probs", draft_probs), ("num_drafts", num_drafts), ("dev_status", dev_status))
    B, W, V = shape
    a = _pack_accept(target_probs.data_ptr(), _ptr(draft_probs), code, B, W, V, draft_tokens.data_ptr(), _ptr(num_drafts),
                     uniform.data_ptr(), accepted.data_ptr(), tokens.data_ptr(), _ptr(dev_status))
    _call("kda_verify_accept", a, _stream(stream))
