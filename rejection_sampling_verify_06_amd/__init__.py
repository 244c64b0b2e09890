"""Batched speculative-decoding verify step on AMD MI355X (gfx950).

A thin Python face of the C library ``libspec_verify.so`` (include/spec_verify.h).
Everything the verify step computes runs in the library's HIP kernels; this
module only checks tensor shapes and passes device pointers and torch's
current stream.  PyTorch supplies device memory and streams.

    v = Verifier(max_batch=256, max_k=8, max_vocab=152064)
    out = v.run(target, draft, draft_tokens, num_draft, temperature, mode, seed=step)
    out["accepted_len"], out["emitted"], out["p_at"], out["q_at"], out["status"]

Around a decode loop's verify call: ``PagedCache`` (the target's keys and
values, with ``paged_attention`` over them) and ``token_logprobs`` (of what
was emitted).

If the library has not been built, every entry point raises ``LibraryMissing``:
there is no fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

from . import _lib
from ._lib import (  # noqa: F401
    SV_F32, SV_BF16, SV_F16, SV_SAMPLE, SV_GREEDY, SV_ONEHOT, SV_STRICT,
    SV_ST_BAD_LAYOUT, SV_ST_K_TOO_LARGE, SV_ST_BAD_MODE, SV_ST_BAD_TEMPERATURE,
    SV_ST_NO_DRAFT_LOGITS, SV_ST_BAD_TOKEN, SV_ST_NONFINITE, SV_ST_ZERO_RESIDUAL,
    SV_ST_BAD_SEQ, SV_ST_BAD_LENGTH, SV_ST_BAD_PAGE, SV_ST_CACHE_FULL,
    KERNEL_NAMES, LibraryMissing,
    SV_ADAPT_WINDOW, SV_ADAPT_MULTIPLICATIVE, SV_ADAPT_OPTIMAL_K, SV_ADAPT_COUNT_EMITTED, SV_ADAPT_COUNT_DRAFT_ONLY,
)

__all__ = ["Verifier", "VerifyError", "verify", "propose_ngram", "NgramProposer", "AcceptanceStats",
           "DraftLengthController", "token_logprobs", "paged_attention", "PagedCache",
           "LibraryMissing", "KERNEL_NAMES"]


class VerifyError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"spec_verify error {code}: {msg}")
        self.code = code


def _check(rc: int):
    if rc != 0:
        raise VerifyError(rc, _lib.last_error())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _logits_dtype(t, torch):
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _need(t, name, dtypes, torch, numel=None, device=None):
    if t is None:
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements, expected {numel}")


class Verifier:
    """One library context (device scratch sized for the given maxima)."""

    def __init__(self, max_batch: int, max_k: int, max_vocab: int, device: Optional[int] = None):
        import torch
        self._torch = torch
        self._lib = _lib.load()
        self.device = torch.cuda.current_device() if device is None else int(device)
        self.max_batch, self.max_k, self.max_vocab = int(max_batch), int(max_k), int(max_vocab)
        h = ctypes.c_void_p()
        _check(self._lib.spec_verify_create(ctypes.byref(h), self.device, self.max_batch, self.max_k,
                                            self.max_vocab))
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.spec_verify_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- outputs ------------------------------------------------------------
    def make_outputs(self, batch: int, total_draft: int, want_pq: bool = True, want_status: bool = True) -> dict:
        torch = self._torch
        dev = torch.device("cuda", self.device)
        return {
            "accepted_len": torch.empty(batch, dtype=torch.int32, device=dev),
            "emitted": torch.empty(total_draft + batch, dtype=torch.int32, device=dev),
            "p_at": torch.empty(total_draft, dtype=torch.float32, device=dev) if want_pq else None,
            "q_at": torch.empty(total_draft, dtype=torch.float32, device=dev) if want_pq else None,
            "status": torch.empty(batch, dtype=torch.int32, device=dev) if want_status else None,
        }

    # -- the step -------------------------------------------------------------
    def build_args(self, target, draft, draft_tokens, num_draft, temperature=None, mode=None, seq_ids=None,
                   seed: int = 0, out: Optional[dict] = None, vocab: Optional[int] = None,
                   total_draft: Optional[int] = None, top_k=None, top_p=None) -> "_lib.SpecVerifyArgs":
        """Check shapes and pack the argument struct (no device work)."""
        torch = self._torch
        dev = torch.device("cuda", self.device)
        if target.dim() != 2 or target.stride(1) != 1:
            raise ValueError("target must be 2-D with unit column stride")
        B = int(num_draft.numel())
        T = int(draft_tokens.numel()) if total_draft is None else int(total_draft)
        V = int(target.shape[1]) if vocab is None else int(vocab)
        if target.shape[0] != T + B:
            raise ValueError(f"target has {target.shape[0]} rows, expected total_draft + B = {T + B}")
        if not target.is_cuda or target.device != dev:
            raise ValueError("target must be on the context's device")
        if draft is not None and draft.numel() == 0:
            draft = None
        if draft is not None:
            if draft.dim() != 2 or draft.stride(1) != 1 or draft.shape[0] != T or not draft.is_cuda:
                raise ValueError("draft must be a 2-D device tensor [total_draft, >= vocab] with unit column stride")
        _need(draft_tokens, "draft_tokens", (torch.int32,), torch, T, dev)
        _need(num_draft, "num_draft", (torch.int32,), torch, B, dev)
        _need(temperature, "temperature", (torch.float32,), torch, B, dev)
        _need(mode, "mode", (torch.uint8,), torch, B, dev)
        _need(seq_ids, "seq_ids", (torch.int32, getattr(torch, "uint32", torch.int32)), torch, B, dev)
        _need(top_k, "top_k", (torch.int32,), torch, B, dev)
        _need(top_p, "top_p", (torch.float32,), torch, B, dev)
        if out is None:
            raise ValueError("out is required (see make_outputs)")
        _need(out["accepted_len"], "accepted_len", (torch.int32,), torch, B, dev)
        _need(out["emitted"], "emitted", (torch.int32,), torch, T + B, dev)
        _need(out.get("p_at"), "p_at", (torch.float32,), torch, T, dev)
        _need(out.get("q_at"), "q_at", (torch.float32,), torch, T, dev)
        _need(out.get("status"), "status", (torch.int32,), torch, B, dev)
        a = _lib.SpecVerifyArgs()
        a.batch = B
        a.vocab = V
        a.total_draft = T
        a.target_dtype = _logits_dtype(target, torch)
        a.draft_dtype = _logits_dtype(draft, torch) if draft is not None else SV_F32
        a.target_logits = target.data_ptr()
        a.ld_target = target.stride(0)
        a.draft_logits = _ptr(draft)
        a.ld_draft = draft.stride(0) if draft is not None else 0
        a.draft_tokens = _ptr(draft_tokens) if T > 0 else None
        a.num_draft = num_draft.data_ptr()
        a.temperature = _ptr(temperature)
        a.mode = _ptr(mode)
        a.seq_ids = _ptr(seq_ids)
        a.seed = int(seed) & 0xFFFFFFFFFFFFFFFF
        a.accepted_len = out["accepted_len"].data_ptr()
        a.emitted_tokens = out["emitted"].data_ptr()
        a.p_at_proposal = _ptr(out.get("p_at"))
        a.q_at_proposal = _ptr(out.get("q_at"))
        a.status = _ptr(out.get("status"))
        a.top_k = _ptr(top_k)
        a.top_p = _ptr(top_p)
        return a

    def run_args(self, args: "_lib.SpecVerifyArgs", stream=None):
        """Enqueue one step from a packed argument struct on ``stream``
        (default: torch's current stream on the context's device)."""
        s = self._torch.cuda.current_stream(self.device) if stream is None else stream
        _check(self._lib.spec_verify_run(self._h, ctypes.byref(args), ctypes.c_void_p(s.cuda_stream)))

    def run(self, target, draft, draft_tokens, num_draft, temperature=None, mode=None, seq_ids=None,
            seed: int = 0, out: Optional[dict] = None, want_pq: bool = True, want_status: bool = True,
            vocab: Optional[int] = None, total_draft: Optional[int] = None, stream=None,
            top_k=None, top_p=None) -> dict:
        if out is None:
            T = int(draft_tokens.numel()) if total_draft is None else int(total_draft)
            out = self.make_outputs(int(num_draft.numel()), T, want_pq, want_status)
        args = self.build_args(target, draft, draft_tokens, num_draft, temperature, mode, seq_ids, seed, out,
                               vocab, total_draft, top_k, top_p)
        self.run_args(args, stream)
        return out

    # -- measurement hooks ------------------------------------------------------
    def timing_enable(self, max_calls: int):
        _check(self._lib.spec_verify_timing_enable(self._h, int(max_calls)))

    def timing_read(self):
        calls = ctypes.c_int32()
        ms = (ctypes.c_double * _lib.SV_NUM_KERNELS)()
        _check(self._lib.spec_verify_timing_read(self._h, ctypes.byref(calls), ms))
        return int(calls.value), dict(zip(KERNEL_NAMES, list(ms)))


_SHARED: dict = {}


def _shared_verifier(dev: int, B: int, kmax: int, V: int) -> Verifier:
    """The one context per device that ``verify`` uses.  It only grows: a
    call beyond its sizes replaces it by one sized for the larger of the old
    and the new maxima (the batch rounded up to a power of two), so a serving
    loop with varying batch sizes holds one context, not one per size."""
    v = _SHARED.get(dev)
    if v is not None and B <= v.max_batch and kmax <= v.max_k and V <= v.max_vocab:
        return v
    nb = 1
    while nb < B:
        nb *= 2
    if v is not None:
        nb, kmax, V = max(nb, v.max_batch), max(kmax, v.max_k), max(V, v.max_vocab)
        import torch
        torch.cuda.synchronize(dev)      # work queued on the old context finishes before its scratch is freed
        v.close()
        del _SHARED[dev]
    v = _SHARED[dev] = Verifier(min(nb, 4096), kmax, V, dev)
    return v


def verify(target, draft, draft_tokens, num_draft, temperature=None, mode=None, seed: int = 0,
           want_pq: bool = False, seq_ids=None, top_k=None, top_p=None, want_status: bool = True) -> dict:
    """One-shot verify step on torch's current stream: allocates the outputs
    (``p_at``/``q_at`` only with ``want_pq``, ``status`` only with
    ``want_status``) and runs the library on a per-device context that is
    reused across calls.  ``top_k`` / ``top_p`` are optional per-sequence
    filters (int32 / float32 [B])."""
    import torch
    dev = target.device.index if target.device.index is not None else torch.cuda.current_device()
    B = int(num_draft.numel())
    T = int(draft_tokens.numel())
    kmax = max(1, min(128, T))          # K_s <= total_draft: the context holds any split of it
    v = _shared_verifier(dev, max(B, 1), kmax, int(target.shape[1]))
    return v.run(target, draft, draft_tokens, num_draft, temperature, mode, seq_ids, seed, want_pq=want_pq,
                 want_status=want_status, top_k=top_k, top_p=top_p)


class NgramProposer:
    """N-gram (prompt-lookup) proposals for a ragged batch of histories
    (spec_verify_ngram_propose).  Holds only its packed argument struct, so a
    caller that reuses the output tensors can re-run it cheaply."""

    def __init__(self):
        self._lib = _lib.load()

    def make_outputs(self, batch: int, max_tokens: int, device, want_match: bool = True) -> dict:
        import torch
        return {"draft_tokens": torch.empty((batch, max_tokens), dtype=torch.int32, device=device),
                "num_draft": torch.empty(batch, dtype=torch.int32, device=device),
                "match_n": torch.empty(batch, dtype=torch.int32, device=device) if want_match else None}

    def build_args(self, history, offsets, min_n: int, max_n: int, max_tokens: int, out: dict):
        import torch
        dev = offsets.device
        B = int(offsets.numel()) - 1
        if B < 0:
            raise ValueError("offsets needs batch + 1 entries")
        _need(offsets, "offsets", (torch.int64,), torch, device=dev)
        _need(history, "history", (torch.int32,), torch, device=dev)
        _need(out["draft_tokens"], "draft_tokens", (torch.int32,), torch, B * max_tokens, dev)
        _need(out["num_draft"], "num_draft", (torch.int32,), torch, B, dev)
        _need(out.get("match_n"), "match_n", (torch.int32,), torch, B, dev)
        a = _lib.SpecVerifyNgramArgs()
        a.batch = B
        a.history = _ptr(history) if history.numel() else None
        a.hist_offsets = _ptr(offsets)
        a.total_len = int(history.numel())
        a.min_n, a.max_n, a.max_tokens = int(min_n), int(max_n), int(max_tokens)
        a.draft_tokens = _ptr(out["draft_tokens"])
        a.num_draft = _ptr(out["num_draft"])
        a.match_n = _ptr(out.get("match_n"))
        return a

    def run_args(self, args, stream=None):
        import torch
        st = stream if stream is not None else torch.cuda.current_stream()
        _check(self._lib.spec_verify_ngram_propose(ctypes.byref(args), ctypes.c_void_p(st.cuda_stream)))

    def run(self, history, offsets, min_n: int = 2, max_n: int = 4, max_tokens: int = 5, stream=None) -> dict:
        B = int(offsets.numel()) - 1
        out = self.make_outputs(B, max_tokens, offsets.device)
        self.run_args(self.build_args(history, offsets, min_n, max_n, max_tokens, out), stream)
        return out


def propose_ngram(history, offsets, min_n: int = 2, max_n: int = 4, max_tokens: int = 5) -> dict:
    """One-shot N-gram proposals: draft_tokens [B, max_tokens] (-1 padded),
    num_draft [B], match_n [B] (0: no occurrence)."""
    return NgramProposer().run(history, offsets, min_n, max_n, max_tokens)


class AcceptanceStats:
    """Acceptance counters kept on the device (spec_verify_stats_accumulate /
    spec_verify_stats_summary).  `counters` is int64 storage for the C
    interface's uint64 words; `add` queues one call's rounds, `summary`
    queues the rates into a float64 tensor."""

    def __init__(self, max_k: int, device):
        import torch
        self._lib = _lib.load()
        self.max_k = int(max_k)
        self.counters = torch.zeros(_lib.stats_words(self.max_k), dtype=torch.int64, device=device)

    def reset(self):
        self.counters.zero_()

    def add(self, num_draft, accepted_len, stream=None):
        import torch
        B = int(num_draft.numel())
        _need(num_draft, "num_draft", (torch.int32,), torch, B, self.counters.device)
        _need(accepted_len, "accepted_len", (torch.int32,), torch, B, self.counters.device)
        st = stream if stream is not None else torch.cuda.current_stream()
        _check(self._lib.spec_verify_stats_accumulate(B, self.max_k, _ptr(num_draft), _ptr(accepted_len),
                                                      _ptr(self.counters), ctypes.c_void_p(st.cuda_stream)))

    def bind(self, num_draft, accepted_len, stream=None):
        """Check the arguments once and return a callable that only queues
        the accumulation (for a caller that reuses the same tensors)."""
        import torch
        B = int(num_draft.numel())
        _need(num_draft, "num_draft", (torch.int32,), torch, B, self.counters.device)
        _need(accepted_len, "accepted_len", (torch.int32,), torch, B, self.counters.device)
        st = ctypes.c_void_p((stream if stream is not None else torch.cuda.current_stream()).cuda_stream)
        f, a = self._lib.spec_verify_stats_accumulate, (B, self.max_k, _ptr(num_draft), _ptr(accepted_len),
                                                       _ptr(self.counters), st)
        return lambda: _check(f(*a))

    def summary(self, out=None, stream=None):
        import torch
        if out is None:
            out = torch.empty(_lib.stats_summary_words(self.max_k), dtype=torch.float64, device=self.counters.device)
        _need(out, "summary", (torch.float64,), torch, _lib.stats_summary_words(self.max_k), self.counters.device)
        st = stream if stream is not None else torch.cuda.current_stream()
        _check(self._lib.spec_verify_stats_summary(self.max_k, _ptr(self.counters), _ptr(out),
                                                   ctypes.c_void_p(st.cuda_stream)))
        return out


class DraftLengthController:
    """Per-sequence draft-length controllers on the device
    (spec_verify_adapt_reset / spec_verify_adapt).  `update` takes a round's
    num_draft and accepted_len and returns the next lengths (int32 [batch]).
    `count` picks the ratio: SV_ADAPT_COUNT_EMITTED (the pages' count,
    min(A + 1, K) / K) or SV_ADAPT_COUNT_DRAFT_ONLY (A / max(K, 1))."""

    def __init__(self, batch: int, kind: int = SV_ADAPT_WINDOW, *, min_k: int = 1, max_k: int = 10,
                 window: int = 100, min_samples: int = 10, target: float = 0.7, rate: float = 0.1,
                 init_k: int = 5, device=None, count: int = SV_ADAPT_COUNT_EMITTED):
        import torch
        self._lib = _lib.load()
        dev = torch.device("cuda", 0) if device is None else torch.device(device)
        self.batch = int(batch)
        nbytes = _lib.adapt_state_bytes(self.batch, window if kind == SV_ADAPT_WINDOW else 0)
        self.state = torch.empty(max(nbytes, 16) // 8 + 1, dtype=torch.int64, device=dev)
        self.next_k = torch.empty(self.batch, dtype=torch.int32, device=dev)
        a = _lib.SpecVerifyAdaptArgs()
        a.batch, a.kind, a.min_k, a.max_k = self.batch, int(kind), int(min_k), int(max_k)
        a.window, a.min_samples, a.target, a.rate = int(window), int(min_samples), float(target), float(rate)
        a.count = int(count)
        a.state, a.next_k = _ptr(self.state), _ptr(self.next_k)
        self._args = a
        self.reset(init_k)

    def reset(self, init_k: int, stream=None):
        import torch
        st = stream if stream is not None else torch.cuda.current_stream()
        _check(self._lib.spec_verify_adapt_reset(ctypes.byref(self._args), int(init_k),
                                                 ctypes.c_void_p(st.cuda_stream)))

    def bind(self, num_draft, accepted_len, stream=None):
        """Check the arguments once and return a callable that only queues
        the update (for a caller that reuses the same tensors)."""
        import torch
        _need(num_draft, "num_draft", (torch.int32,), torch, self.batch, self.next_k.device)
        _need(accepted_len, "accepted_len", (torch.int32,), torch, self.batch, self.next_k.device)
        a = _lib.SpecVerifyAdaptArgs()
        ctypes.pointer(a)[0] = self._args
        a.num_draft, a.accepted_len = _ptr(num_draft), _ptr(accepted_len)
        st = ctypes.c_void_p((stream if stream is not None else torch.cuda.current_stream()).cuda_stream)
        f, ref = self._lib.spec_verify_adapt, ctypes.byref(a)
        return lambda: _check(f(ref, st))

    def update(self, num_draft, accepted_len, stream=None):
        import torch
        _need(num_draft, "num_draft", (torch.int32,), torch, self.batch, self.next_k.device)
        _need(accepted_len, "accepted_len", (torch.int32,), torch, self.batch, self.next_k.device)
        self._args.num_draft, self._args.accepted_len = _ptr(num_draft), _ptr(accepted_len)
        st = stream if stream is not None else torch.cuda.current_stream()
        _check(self._lib.spec_verify_adapt(ctypes.byref(self._args), ctypes.c_void_p(st.cuda_stream)))
        return self.next_k


def _int32(v, name) -> int:
    """An argument of the C interface that is an int32 (ctypes would wrap it)."""
    v = int(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name} {v} does not fit 32 bits")
    return v


_AS_IT_IS = contextlib.nullcontext()


def _on_stream(dev, stream, *inputs):
    """A context in which a call's stream is torch's current one (so that what
    the call allocates belongs to it) and its device the current device.  On a
    stream that is given, the inputs may have been allocated on another one:
    their memory is kept until this one has passed the call."""
    import torch
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        return torch.cuda.stream(stream)
    return _AS_IT_IS if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _for_caller(out, dev, stream):
    """The outputs of a call on a stream that was given: allocated there, and
    kept until the stream the caller works on has passed its use of them."""
    if stream is not None:
        import torch
        caller = torch.cuda.current_stream(dev)
        for t in out.values() if isinstance(out, dict) else (out,):
            if t is not None:
                t.record_stream(caller)
    return out


def _queue(dev) -> int:
    """The handle of torch's current stream on a device."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev.index)


def token_logprobs(logits, tokens=None, *, top: int = 0, temperature=None, vocab: Optional[int] = None,
                   want_entropy: bool = True, want_rank: bool = True, want_status: bool = True, stream=None) -> dict:
    """Log probabilities of one given token per row of ``logits`` ([rows, >=
    vocab], float32 or bfloat16, unit column stride), with entropy, rank and
    the ``top`` best alternatives (spec_verify_token_logprobs).

    ``tokens`` is int32 [rows]; a negative token leaves its row out, so a
    verify call's ``emitted`` goes with its ``target`` as they are.  Without
    ``tokens`` every row is read, for entropy and alternatives alone.
    ``temperature`` is float32 [rows].  Returns ``logprob``, ``entropy``
    (float32 [rows]), ``rank`` (int32 [rows], 1 for the largest logit),
    ``top_tokens`` (int32 [rows, top]), ``top_logprobs`` (float32 [rows,
    top]) and ``status`` (int32 [rows]); what was not asked for is None,
    except the empty [rows, 0] alternatives of ``top`` = 0."""
    import torch
    lib = _lib.load()
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-D with unit column stride")
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    dev = logits.device
    R, V = int(logits.shape[0]), int(logits.shape[1]) if vocab is None else int(vocab)
    if V < 1 or V > logits.shape[1]:
        raise ValueError(f"vocab {V} outside 1..{logits.shape[1]} columns")
    dtype = _logits_dtype(logits, torch)
    _need(tokens, "tokens", (torch.int32,), torch, R, dev)
    _need(temperature, "temperature", (torch.float32,), torch, R, dev)
    top = _int32(top, "top")
    nbytes = lib.spec_verify_logprobs_workspace(R, V, dtype, top)
    if nbytes < 0:
        _check(int(nbytes))
    with _on_stream(dev, stream, logits, tokens, temperature):
        f32, i32 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.int32, device=dev)
        out = {
            "logprob": torch.empty(R, **f32) if tokens is not None else None,
            "entropy": torch.empty(R, **f32) if want_entropy else None,
            "rank": torch.empty(R, **i32) if want_rank and tokens is not None else None,
            "top_tokens": torch.empty((R, top), **i32),
            "top_logprobs": torch.empty((R, top), **f32),
            "status": torch.empty(R, **i32) if want_status else None,
        }
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        a = _lib.SpecVerifyLogprobsArgs(
            R, V, dtype, top, logits.data_ptr(), logits.stride(0) if R > 1 else logits.shape[1], _ptr(tokens),
            _ptr(temperature), _ptr(out["logprob"]), _ptr(out["entropy"]), _ptr(out["rank"]),
            out["top_tokens"].data_ptr() if top else None, out["top_logprobs"].data_ptr() if top else None,
            _ptr(out["status"]), ws.data_ptr(), nbytes)
        _check(lib.spec_verify_token_logprobs(ctypes.byref(a), _queue(dev)))
    return _for_caller(out, dev, stream)


def _cache_dtype(t, name, torch):
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float16:
        return SV_F16
    raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")


def paged_attention(q, k_pages, v_pages, page_table, seq_len, num_draft, *, seqs=None, scale: Optional[float] = None,
                    window: int = 0, want_lse: bool = False, want_status: bool = True, stream=None, start=None) -> dict:
    """Attention of a round's new tokens over a paged key-value cache
    (spec_verify_paged_attention).

    ``q`` is [total_rows, heads, head_dim], bfloat16 or float16: for each
    sequence its ``num_draft`` + 1 rows, packed like a verify call's target
    rows (``num_draft`` 0: one new token).  ``k_pages`` / ``v_pages`` are
    [num_pages, kv_heads, page_size, head_dim] (any strides of the first
    three), ``page_table`` int32 [slots, max_pages], ``seq_len`` int32
    [slots]: the cached tokens, the new ones last.  Sequence b uses slot
    ``seqs[b]`` (int32), or b.  Row i sees positions up to seq_len -
    num_draft - 1 + i, with ``window`` > 0 only the last ``window`` of them.
    ``scale`` defaults to head_dim ** -0.5.  ``start`` (int32 [batch], from
    ``PagedCache.reserve``): a sequence whose reserve was refused has no new
    tokens, and gets NaN and a status.  Returns ``out`` like ``q``
    (contiguous), ``lse`` (float32 [total_rows, heads]) and ``status`` (int32
    [batch]); what was not asked for is None."""
    import torch
    lib = _lib.load()
    if q.dim() != 3 or k_pages.dim() != 4 or v_pages.shape != k_pages.shape or page_table.dim() != 2:
        raise ValueError("q must be 3-D, k_pages and v_pages 4-D of one shape, page_table 2-D")
    dev = q.device
    N, H, D = q.shape
    pages, KV, P, Dk = k_pages.shape
    if D != Dk:
        raise ValueError(f"q has head_dim {D}, the pages {Dk}")
    if k_pages.dtype != q.dtype or v_pages.dtype != q.dtype:
        raise TypeError(f"q is {q.dtype}, the pages {k_pages.dtype} and {v_pages.dtype}")
    if not q.is_cuda or k_pages.device != dev or v_pages.device != dev:
        raise ValueError(f"q, k_pages and v_pages must be on one GPU, got {dev}, {k_pages.device} and {v_pages.device}")
    qs, ks, vs = q.stride(), k_pages.stride(), v_pages.stride()
    if qs[2] != 1 or ks[3] != 1 or vs[3] != 1:
        raise ValueError("q, k_pages and v_pages must have unit stride in their last dimension")
    _need(num_draft, "num_draft", (torch.int32,), torch, None, dev)
    B, (slots, width), ts = num_draft.numel(), page_table.shape, page_table.stride()
    _need(seqs, "seqs", (torch.int32,), torch, B, dev)
    _need(start, "start", (torch.int32,), torch, B, dev)
    _need(seq_len, "seq_len", (torch.int32,), torch, slots, dev)
    if page_table.dtype != torch.int32 or page_table.device != dev or (width > 1 and ts[1] != 1):
        raise ValueError("page_table must be int32 on q's device with unit column stride")
    if seqs is None and B > slots:
        raise ValueError(f"{B} sequences, but page_table has {slots} rows")
    a = _lib.SpecVerifyAttentionArgs(
        B, N, H, KV, D, _cache_dtype(q, "q", torch), P, _int32(window, "window"), pages, slots, width,
        ts[0] if slots > 1 else width,
        # strides of dimensions of size 1 say nothing
        q.data_ptr(), qs[0] if N > 1 else 0, qs[1] if H > 1 else 0,
        k_pages.data_ptr(), ks[0] if pages > 1 else 0, ks[1] if KV > 1 else 0, ks[2],
        v_pages.data_ptr(), vs[0] if pages > 1 else 0, vs[1] if KV > 1 else 0, vs[2],
        page_table.data_ptr(), seq_len.data_ptr(), _ptr(seqs), num_draft.data_ptr(),
        D ** -0.5 if scale is None else float(scale), start=_ptr(start))
    nbytes = lib.spec_verify_attention_workspace(ctypes.byref(a))
    if nbytes < 0:
        _check(int(nbytes))
    with _on_stream(dev, stream, q, k_pages, v_pages, page_table, seq_len, num_draft, seqs, start):
        out = {
            "out": torch.empty((N, H, D), dtype=q.dtype, device=dev),
            "lse": torch.empty((N, H), dtype=torch.float32, device=dev) if want_lse else None,
            "status": torch.empty(B, dtype=torch.int32, device=dev) if want_status else None,
        }
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        a.out, a.lse, a.status = out["out"].data_ptr(), _ptr(out["lse"]), _ptr(out["status"])
        a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
        _check(lib.spec_verify_paged_attention(ctypes.byref(a), _queue(dev)))
    return _for_caller(out, dev, stream)


class PagedCache:
    """A paged key-value cache on the device (spec_verify_cache_*): ``k`` and
    ``v`` [layers, num_pages, kv_heads, page_size, head_dim], ``page_table``
    int32 [max_seqs, max_pages] (-1 behind a sequence's pages), ``seq_len``
    int32 [max_seqs], ``refcount`` int32 [num_pages] (0: free).

    A round of speculative decoding over it:

        r = cache.reserve(seqs, num_draft + 1, total)      # places for the new tokens
        cache.write(layer, k_new, v_new, r["slots"])       # every layer, before it attends
        o = cache.attend(layer, q, num_draft, seqs, start=r["start"])
        ...                                                # logits, Verifier.run
        cache.commit(seqs, num_draft, out["accepted_len"], start=r["start"])   # the rejected tokens leave

    ``seqs`` (int32 [batch], distinct slots, or None for 0 .. batch - 1) and
    the counts are device tensors; nothing here waits for the device.  The
    calls return a status per entry (0, or SV_ST_* bits of why it was refused
    and changed nothing).  With ``start`` a sequence that could not be reserved
    for sits its round out: its rows of ``o`` are NaN, so that a verify call
    over their logits refuses it, and ``commit`` leaves it as it was.  Calls on
    one cache must be ordered on one stream."""

    def __init__(self, layers: int, num_pages: int, page_size: int, kv_heads: int, head_dim: int, max_seqs: int,
                 max_pages: int, dtype=None, device=None):
        import torch
        self._torch, self._lib = torch, _lib.load()
        dtype = torch.bfloat16 if dtype is None else dtype
        dev = torch.device("cuda", 0) if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"the cache lives on a GPU, not on {dev}")
        dev = torch.device("cuda", torch.cuda.current_device()) if dev.index is None else dev
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"cached keys and values are bfloat16 or float16, got {dtype}")
        c = _lib.SpecVerifyCache(*(_int32(v, name) for v, name in (
            (max_seqs, "max_seqs"), (max_pages, "max_pages"), (page_size, "page_size"), (num_pages, "num_pages"),
            (layers, "layers"), (kv_heads, "kv_heads"), (head_dim, "head_dim"))))
        nbytes = self._lib.spec_verify_cache_workspace(ctypes.byref(c))
        if nbytes < 0:
            _check(int(nbytes))
        self.device, self.layers, self.page_size = dev, int(layers), int(page_size)
        shape = (c.layers, c.num_pages, c.kv_heads, c.page_size, c.head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=dev)
        self.v = torch.empty(shape, dtype=dtype, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        self.page_table = torch.full((c.slots, c.max_pages), -1, **i32)
        self.seq_len = torch.zeros(c.slots, **i32)
        self.refcount = torch.zeros(c.num_pages, **i32)
        self._ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        c.page_table, c.seq_len, c.refcount = _ptr(self.page_table), _ptr(self.seq_len), _ptr(self.refcount)
        c.k, c.v, c.workspace, c.workspace_bytes = _ptr(self.k), _ptr(self.v), _ptr(self._ws), nbytes
        self._c, self._heads = c, (c.kv_heads, c.head_dim)
        self._ref = ctypes.byref(c)

    def _on_stream(self, stream, *inputs):
        if stream is None:
            return _on_stream(self.device, None)
        return _on_stream(self.device, stream, self.k, self.v, self.page_table, self.seq_len, self.refcount, self._ws, *inputs)

    def _entries(self, seqs, counts, name):
        """The batch size, with the index arrays checked."""
        torch = self._torch
        _need(counts, name, (torch.int32,), torch, None, self.device)
        B = int(counts.numel())
        _need(seqs, "seqs", (torch.int32,), torch, B, self.device)
        return B

    def reserve(self, seqs, num_new, total_new: int, stream=None) -> dict:
        """Grows each sequence by ``num_new`` tokens (int32 [batch], summing to
        ``total_new``).  Returns ``start`` (int32 [batch]: the old lengths),
        ``slots`` (int64 [total_new]: the new tokens' places, for ``write``)
        and ``status``; -1 in the first two where an entry was refused.  Users
        of a partly filled last page that all append in one call each get a
        copy of it, and it is free only afterwards: one page more than in two
        calls."""
        torch = self._torch
        B, n = self._entries(seqs, num_new, "num_new"), int(total_new)
        with self._on_stream(stream, seqs, num_new):
            out = {"start": torch.empty(B, dtype=torch.int32, device=self.device),
                   "slots": torch.empty(max(n, 0), dtype=torch.int64, device=self.device),
                   "status": torch.empty(B, dtype=torch.int32, device=self.device)}
            _check(self._lib.spec_verify_cache_reserve(self._ref, B, _ptr(seqs), num_new.data_ptr(), n, _ptr(out["start"]),
                                                       _ptr(out["slots"]), _ptr(out["status"]), _queue(self.device)))
        return _for_caller(out, self.device, stream)

    def write(self, layer: int, k_new, v_new, slots, stream=None):
        """Puts rows of ``k_new`` / ``v_new`` ([rows, kv_heads, head_dim], unit
        stride in head_dim) into the places ``slots`` of ``reserve``."""
        rows, dev, heads = slots.numel(), self.device, self._heads
        _need(slots, "slots", (self._torch.int64,), self._torch, None, dev)
        for t, name in ((k_new, "k_new"), (v_new, "v_new")):
            if t.shape != (rows, *heads) or t.stride(2) != 1:
                raise ValueError(f"{name} must be [{rows}, {heads[0]}, {heads[1]}] with unit stride in the last dimension, got "
                                 f"{tuple(t.shape)}")
            if t.dtype != self.k.dtype:
                raise TypeError(f"{name} is {t.dtype}, the cache {self.k.dtype}")
            if t.device != dev:
                raise ValueError(f"{name} is on {t.device}, the cache on {dev}")
        # strides of dimensions of size 1 say nothing
        r, h = rows > 1, heads[0] > 1
        with self._on_stream(stream, k_new, v_new, slots):
            _check(self._lib.spec_verify_cache_write(
                self._ref, _int32(layer, "layer"), rows, k_new.data_ptr(), k_new.stride(0) if r else 0, k_new.stride(1) if h else 0,
                v_new.data_ptr(), v_new.stride(0) if r else 0, v_new.stride(1) if h else 0, slots.data_ptr(), _queue(dev)))

    def attend(self, layer: int, q, num_draft, seqs=None, **kw) -> dict:
        """``paged_attention`` of ``q`` over a layer of this cache."""
        if not 0 <= int(layer) < self.layers:
            raise ValueError(f"layer {layer} outside 0..{self.layers - 1}")
        return paged_attention(q, self.k[layer], self.v[layer], self.page_table, self.seq_len, num_draft, seqs=seqs, **kw)

    def commit(self, seqs, num_draft, accepted_len, stream=None, *, start=None):
        """Keeps ``accepted_len`` + 1 of the ``num_draft`` + 1 tokens each
        sequence reserved for its round (none where it is -1: not verified).
        With ``start`` (int32 [batch], from ``reserve``) a sequence whose
        reserve was refused keeps what it has; without, every one of them has
        to have been carried out."""
        torch = self._torch
        B = self._entries(seqs, num_draft, "num_draft")
        _need(accepted_len, "accepted_len", (torch.int32,), torch, B, self.device)
        _need(start, "start", (torch.int32,), torch, B, self.device)
        with self._on_stream(stream, seqs, num_draft, accepted_len, start):
            status = torch.empty(B, dtype=torch.int32, device=self.device)
            a = (self._ref, B, _ptr(seqs), num_draft.data_ptr(), accepted_len.data_ptr())
            if start is None:
                _check(self._lib.spec_verify_cache_commit(*a, _ptr(status), _queue(self.device)))
            else:
                _check(self._lib.spec_verify_cache_commit_reserved(*a, _ptr(start), _ptr(status), _queue(self.device)))
        return _for_caller(status, self.device, stream)

    def truncate(self, seqs, drop, stream=None):
        """Takes the last ``drop`` tokens (int32 [batch]) off each sequence."""
        torch = self._torch
        B = self._entries(seqs, drop, "drop")
        with self._on_stream(stream, seqs, drop):
            status = torch.empty(B, dtype=torch.int32, device=self.device)
            _check(self._lib.spec_verify_cache_truncate(self._ref, B, _ptr(seqs), drop.data_ptr() if B else None,
                                                        _ptr(status), _queue(self.device)))
        return _for_caller(status, self.device, stream)

    def release(self, seqs, stream=None):
        """Empties the sequences (int32 [batch])."""
        torch = self._torch
        B = self._entries(None, seqs, "seqs")
        with self._on_stream(stream, seqs):
            status = torch.empty(B, dtype=torch.int32, device=self.device)
            _check(self._lib.spec_verify_cache_truncate(self._ref, B, seqs.data_ptr(), None, _ptr(status), _queue(self.device)))
        return _for_caller(status, self.device, stream)

    def fork(self, parents, children, stream=None):
        """The empty slots ``children`` share everything ``parents`` hold (both
        int32 [batch]; a parent may be named more than once)."""
        torch = self._torch
        B = self._entries(children, parents, "parents")
        with self._on_stream(stream, parents, children):
            status = torch.empty(B, dtype=torch.int32, device=self.device)
            _check(self._lib.spec_verify_cache_fork(self._ref, B, parents.data_ptr(), children.data_ptr(), _ptr(status),
                                                    _queue(self.device)))
        return _for_caller(status, self.device, stream)

    def compact(self, stream=None):
        """Moves the pages in use to the front of the pool; returns their
        number (int32 [1]).  ``slots`` handed out before are void."""
        torch = self._torch
        with self._on_stream(stream):
            live = torch.empty(1, dtype=torch.int32, device=self.device)
            _check(self._lib.spec_verify_cache_compact(self._ref, live.data_ptr(), _queue(self.device)))
        return _for_caller(live, self.device, stream)


def library_loaded_path() -> str:
    """Path of the loaded library (raises LibraryMissing if not built)."""
    _lib.load()
    return _lib.library_path()
