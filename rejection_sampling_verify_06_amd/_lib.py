"""ctypes view of the C interface in include/spec_verify.h (marshalling only)."""
from __future__ import annotations

import ctypes
import os

from .build import library_path

# values from include/spec_verify.h
SV_F32, SV_BF16, SV_F16 = 0, 1, 2
SV_SAMPLE, SV_GREEDY, SV_ONEHOT, SV_STRICT = 0, 1, 2, 3
SV_OK, SV_ERR_INVALID, SV_ERR_NOMEM, SV_ERR_HIP, SV_ERR_CAPACITY = 0, -1, -2, -3, -4
SV_ST_BAD_LAYOUT = 1
SV_ST_K_TOO_LARGE = 2
SV_ST_BAD_MODE = 4
SV_ST_BAD_TEMPERATURE = 8
SV_ST_NO_DRAFT_LOGITS = 16
SV_ST_BAD_TOKEN = 32
SV_ST_NONFINITE = 64
SV_ST_ZERO_RESIDUAL = 128
SV_ST_BAD_SEQ = 256
SV_ST_BAD_LENGTH = 512
SV_ST_BAD_PAGE = 1024
SV_ST_CACHE_FULL = 2048
SV_NUM_KERNELS = 4
KERNEL_NAMES = ("row_stats", "filter", "final", "select")

SV_NGRAM_MAX_N = 16
SV_NGRAM_MAX_TOKENS = 128

SV_STATS_MAX_K = 128
SV_ADAPT_WINDOW, SV_ADAPT_MULTIPLICATIVE, SV_ADAPT_OPTIMAL_K = 0, 1, 2
SV_ADAPT_COUNT_EMITTED, SV_ADAPT_COUNT_DRAFT_ONLY = 0, 1
SV_ADAPT_MAX_WINDOW = 256
SV_ADAPT_MAX_LENGTH = 4096


def stats_words(max_k: int) -> int:
    return 8 + 3 * max_k


def stats_summary_words(max_k: int) -> int:
    return 4 + 2 * max_k


def adapt_state_bytes(batch: int, window: int) -> int:
    return batch * (16 + 8 * window)

EXPORTED = (
    "spec_verify_create", "spec_verify_run", "spec_verify_destroy", "spec_verify_last_error",
    "spec_verify_timing_enable", "spec_verify_timing_read", "spec_verify_version",
    "spec_verify_args_size", "spec_verify_ngram_propose", "spec_verify_ngram_args_size",
    "spec_verify_stats_accumulate", "spec_verify_stats_summary", "spec_verify_adapt_reset", "spec_verify_adapt",
    "spec_verify_adapt_args_size", "spec_verify_run_noalloc",
    "spec_verify_token_logprobs", "spec_verify_logprobs_workspace", "spec_verify_logprobs_args_size",
    "spec_verify_paged_attention", "spec_verify_attention_workspace", "spec_verify_attention_args_size",
    "spec_verify_cache_reserve", "spec_verify_cache_truncate", "spec_verify_cache_commit",
    "spec_verify_cache_commit_reserved", "spec_verify_cache_fork", "spec_verify_cache_compact", "spec_verify_cache_write",
    "spec_verify_cache_workspace", "spec_verify_cache_size",
)
SV_CACHE_MAX_SLOTS = 4096
SV_LOGPROBS_MAX_TOP = 64
SV_NOALLOC_SCRATCH_BYTES = 67108864


class SpecVerifyArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("vocab", ctypes.c_int64),
        ("total_draft", ctypes.c_int64),
        ("target_dtype", ctypes.c_int32),
        ("draft_dtype", ctypes.c_int32),
        ("target_logits", ctypes.c_void_p),
        ("ld_target", ctypes.c_int64),
        ("draft_logits", ctypes.c_void_p),
        ("ld_draft", ctypes.c_int64),
        ("draft_tokens", ctypes.c_void_p),
        ("num_draft", ctypes.c_void_p),
        ("temperature", ctypes.c_void_p),
        ("mode", ctypes.c_void_p),
        ("seq_ids", ctypes.c_void_p),
        ("seed", ctypes.c_uint64),
        ("accepted_len", ctypes.c_void_p),
        ("emitted_tokens", ctypes.c_void_p),
        ("p_at_proposal", ctypes.c_void_p),
        ("q_at_proposal", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("top_k", ctypes.c_void_p),
        ("top_p", ctypes.c_void_p),
    ]


class SpecVerifyNgramArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("history", ctypes.c_void_p),
        ("hist_offsets", ctypes.c_void_p),
        ("total_len", ctypes.c_int64),
        ("min_n", ctypes.c_int32),
        ("max_n", ctypes.c_int32),
        ("max_tokens", ctypes.c_int32),
        ("draft_tokens", ctypes.c_void_p),
        ("num_draft", ctypes.c_void_p),
        ("match_n", ctypes.c_void_p),
    ]


class SpecVerifyAdaptArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("kind", ctypes.c_int32),
        ("min_k", ctypes.c_int32),
        ("max_k", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("min_samples", ctypes.c_int32),
        ("count", ctypes.c_int32),
        ("target", ctypes.c_double),
        ("rate", ctypes.c_double),
        ("num_draft", ctypes.c_void_p),
        ("accepted_len", ctypes.c_void_p),
        ("state", ctypes.c_void_p),
        ("next_k", ctypes.c_void_p),
    ]


class SpecVerifyLogprobsArgs(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("top", ctypes.c_int32),
        ("logits", ctypes.c_void_p),
        ("ld", ctypes.c_int64),
        ("tokens", ctypes.c_void_p),
        ("temperature", ctypes.c_void_p),
        ("logprob", ctypes.c_void_p),
        ("entropy", ctypes.c_void_p),
        ("rank", ctypes.c_void_p),
        ("top_tokens", ctypes.c_void_p),
        ("top_logprobs", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_int64),
    ]


class SpecVerifyAttentionArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("total_rows", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("slots", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int64),
        ("q", ctypes.c_void_p),
        ("q_row_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("k", ctypes.c_void_p),
        ("k_page_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("k_token_stride", ctypes.c_int64),
        ("v", ctypes.c_void_p),
        ("v_page_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("page_table", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p),
        ("seqs", ctypes.c_void_p),
        ("num_draft", ctypes.c_void_p),
        ("scale", ctypes.c_double),
        ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_int64),
        ("start", ctypes.c_void_p),
    ]


class SpecVerifyCache(ctypes.Structure):
    _fields_ = [
        ("slots", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("layers", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_table", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p),
        ("refcount", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_int64),
    ]


_LIB = None


class LibraryMissing(RuntimeError):
    pass


def load() -> ctypes.CDLL:
    """Load libspec_verify.so.  torch is imported first so that the library
    binds to the HIP runtime torch already loaded (one runtime per process,
    so torch's stream handles are valid in the library)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    import torch  # noqa: F401  (loads torch's HIP runtime first)
    path = library_path()
    if not os.path.exists(path):
        raise LibraryMissing(f"{path} is not built; run __graft_entry__.build() (hipcc for gfx950)")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    lib.spec_verify_create.argtypes = [ctypes.POINTER(P), ctypes.c_int, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64]
    lib.spec_verify_create.restype = ctypes.c_int
    lib.spec_verify_run.argtypes = [P, ctypes.POINTER(SpecVerifyArgs), P]
    lib.spec_verify_run.restype = ctypes.c_int
    lib.spec_verify_run_noalloc.argtypes = [ctypes.POINTER(SpecVerifyArgs), ctypes.c_int32, P]
    lib.spec_verify_run_noalloc.restype = ctypes.c_int
    lib.spec_verify_destroy.argtypes = [P]
    lib.spec_verify_destroy.restype = None
    lib.spec_verify_last_error.argtypes = []
    lib.spec_verify_last_error.restype = ctypes.c_char_p
    lib.spec_verify_timing_enable.argtypes = [P, ctypes.c_int32]
    lib.spec_verify_timing_enable.restype = ctypes.c_int
    lib.spec_verify_timing_read.argtypes = [P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_double)]
    lib.spec_verify_timing_read.restype = ctypes.c_int
    lib.spec_verify_version.argtypes = []
    lib.spec_verify_version.restype = ctypes.c_char_p
    lib.spec_verify_args_size.argtypes = []
    lib.spec_verify_args_size.restype = ctypes.c_int64
    lib.spec_verify_ngram_propose.argtypes = [ctypes.POINTER(SpecVerifyNgramArgs), P]
    lib.spec_verify_ngram_propose.restype = ctypes.c_int
    lib.spec_verify_ngram_args_size.argtypes = []
    lib.spec_verify_ngram_args_size.restype = ctypes.c_int64
    lib.spec_verify_stats_accumulate.argtypes = [ctypes.c_int32, ctypes.c_int32, P, P, P, P]
    lib.spec_verify_stats_accumulate.restype = ctypes.c_int
    lib.spec_verify_stats_summary.argtypes = [ctypes.c_int32, P, P, P]
    lib.spec_verify_stats_summary.restype = ctypes.c_int
    lib.spec_verify_adapt_reset.argtypes = [ctypes.POINTER(SpecVerifyAdaptArgs), ctypes.c_int32, P]
    lib.spec_verify_adapt_reset.restype = ctypes.c_int
    lib.spec_verify_adapt.argtypes = [ctypes.POINTER(SpecVerifyAdaptArgs), P]
    lib.spec_verify_adapt.restype = ctypes.c_int
    lib.spec_verify_adapt_args_size.argtypes = []
    lib.spec_verify_adapt_args_size.restype = ctypes.c_int64
    lib.spec_verify_token_logprobs.argtypes = [ctypes.POINTER(SpecVerifyLogprobsArgs), P]
    lib.spec_verify_token_logprobs.restype = ctypes.c_int
    lib.spec_verify_logprobs_workspace.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
    lib.spec_verify_logprobs_workspace.restype = ctypes.c_int64
    lib.spec_verify_logprobs_args_size.argtypes = []
    lib.spec_verify_logprobs_args_size.restype = ctypes.c_int64
    lib.spec_verify_paged_attention.argtypes = [ctypes.POINTER(SpecVerifyAttentionArgs), P]
    lib.spec_verify_paged_attention.restype = ctypes.c_int
    lib.spec_verify_attention_workspace.argtypes = [ctypes.POINTER(SpecVerifyAttentionArgs)]
    lib.spec_verify_attention_workspace.restype = ctypes.c_int64
    lib.spec_verify_attention_args_size.argtypes = []
    lib.spec_verify_attention_args_size.restype = ctypes.c_int64
    C, i32, i64 = ctypes.POINTER(SpecVerifyCache), ctypes.c_int32, ctypes.c_int64
    for name, types in (("reserve", [C, i32, P, P, i64, P, P, P, P]), ("truncate", [C, i32, P, P, P, P]),
                        ("commit", [C, i32, P, P, P, P, P]), ("commit_reserved", [C, i32, P, P, P, P, P, P]),
                        ("fork", [C, i32, P, P, P, P]), ("compact", [C, P, P]),
                        ("write", [C, i32, i64, P, i64, i64, P, i64, i64, P, P])):
        f = getattr(lib, "spec_verify_cache_" + name)
        f.argtypes, f.restype = types, ctypes.c_int
    lib.spec_verify_cache_workspace.argtypes = [C]
    lib.spec_verify_cache_workspace.restype = ctypes.c_int64
    lib.spec_verify_cache_size.argtypes = []
    lib.spec_verify_cache_size.restype = ctypes.c_int64
    if lib.spec_verify_args_size() != ctypes.sizeof(SpecVerifyArgs):
        raise RuntimeError("spec_verify_args layout differs between the library and the binding")
    if lib.spec_verify_ngram_args_size() != ctypes.sizeof(SpecVerifyNgramArgs):
        raise RuntimeError("spec_verify_ngram_args layout differs between the library and the binding")
    if lib.spec_verify_adapt_args_size() != ctypes.sizeof(SpecVerifyAdaptArgs):
        raise RuntimeError("spec_verify_adapt_args layout differs between the library and the binding")
    if lib.spec_verify_logprobs_args_size() != ctypes.sizeof(SpecVerifyLogprobsArgs):
        raise RuntimeError("spec_verify_logprobs_args layout differs between the library and the binding")
    if lib.spec_verify_attention_args_size() != ctypes.sizeof(SpecVerifyAttentionArgs):
        raise RuntimeError("spec_verify_attention_args layout differs between the library and the binding")
    if lib.spec_verify_cache_size() != ctypes.sizeof(SpecVerifyCache):
        raise RuntimeError("spec_verify_cache layout differs between the library and the binding")
    _LIB = lib
    return lib


def last_error() -> str:
    return load().spec_verify_last_error().decode(errors="replace")
