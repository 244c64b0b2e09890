"""CPU checks of the C-ABI library: it builds, loads next to torch's HIP
runtime, exports every function the header declares, and its struct layout
and constants match the binding.  No device calls."""
import ctypes
import os
import re

import pytest
import torch  # noqa: F401  (torch's HIP runtime must be the first one loaded, as in the binding)

from rejection_sampling_verify_06_amd import build as svbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "spec_verify.h")


def _ensure_built():
    if not os.path.exists(svbuild.library_path()):
        svbuild.build_library()
    return svbuild.library_path()


def _declared_functions():
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(spec_verify_[a-z_]+)\s*\(", src)))


def _header_enums():
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    out = {}
    for body in re.findall(r"enum\s*\{(.*?)\}", src, flags=re.S):
        for name, val in re.findall(r"(SV_[A-Z0-9_]+)\s*=\s*(-?\d+)", body):
            out[name] = int(val)
    for name, val in re.findall(r"#define\s+(SV_[A-Z_]+)\s+(\d+)\b", src):
        out[name] = int(val)
    return out


def test_header_declares_the_core_entry_points():
    names = _declared_functions()
    for n in ("spec_verify_create", "spec_verify_run", "spec_verify_destroy", "spec_verify_last_error"):
        assert n in names


def test_library_exports_every_declared_function():
    lib = ctypes.CDLL(_ensure_built())
    missing = [n for n in _declared_functions() if not hasattr(lib, n)]
    assert not missing, missing


def test_binding_knows_every_export():
    from rejection_sampling_verify_06_amd import _lib
    assert sorted(_lib.EXPORTED) == _declared_functions()


def test_struct_layout_and_single_hip_runtime():
    _ensure_built()
    from rejection_sampling_verify_06_amd import _lib
    lib = _lib.load()                       # checks sizeof(spec_verify_args) against the binding
    assert lib.spec_verify_args_size() == ctypes.sizeof(_lib.SpecVerifyArgs) == 168   # with the two filter pointers
    assert lib.spec_verify_adapt_args_size() == ctypes.sizeof(_lib.SpecVerifyAdaptArgs) == 80
    assert b"gfx950" in lib.spec_verify_version()
    maps = open("/proc/self/maps").read()
    hip = {line.split()[-1] for line in maps.splitlines() if "libamdhip64" in line}
    assert len(hip) == 1, hip


def test_constants_match_header():
    from rejection_sampling_verify_06_amd import _lib
    import oracle
    enums = _header_enums()
    for name, val in enums.items():
        if hasattr(_lib, name):
            assert getattr(_lib, name) == val, name
    # the oracle's own copies of the interface encoding
    assert (oracle.SAMPLE, oracle.GREEDY, oracle.ONEHOT) == (enums["SV_SAMPLE"], enums["SV_GREEDY"], enums["SV_ONEHOT"])
    for o, h in (("ST_BAD_LAYOUT", "SV_ST_BAD_LAYOUT"), ("ST_K_TOO_LARGE", "SV_ST_K_TOO_LARGE"),
                 ("ST_BAD_MODE", "SV_ST_BAD_MODE"), ("ST_BAD_TEMPERATURE", "SV_ST_BAD_TEMPERATURE"),
                 ("ST_NO_DRAFT_LOGITS", "SV_ST_NO_DRAFT_LOGITS"), ("ST_BAD_TOKEN", "SV_ST_BAD_TOKEN"),
                 ("ST_NONFINITE", "SV_ST_NONFINITE"), ("ST_ZERO_RESIDUAL", "SV_ST_ZERO_RESIDUAL")):
        assert getattr(oracle, o) == enums[h], o


def test_missing_library_fails_loudly(monkeypatch, tmp_path):
    from rejection_sampling_verify_06_amd import _lib
    monkeypatch.setattr(_lib, "_LIB", None)
    monkeypatch.setattr(_lib, "library_path", lambda: str(tmp_path / "nope.so"))
    with pytest.raises(_lib.LibraryMissing):
        _lib.load()


def test_package_does_not_import_the_oracle():
    """The product package never reaches for the CPU oracle."""
    pkg = os.path.join(ROOT, "rejection_sampling_verify_06_amd")
    for dirpath, _, files in os.walk(pkg):
        for f in files:
            if f.endswith((".py", ".hip", ".cpp", ".h", ".hpp")):
                src = open(os.path.join(dirpath, f)).read()
                assert not re.search(r"^\s*(from|import)\s+oracle\b", src, flags=re.M), f
                assert "workloads" not in src or f.endswith(".md"), f


# ---- host-side argument checks that return before any HIP call (no device needed) ----

def _lib_loaded():
    _ensure_built()
    from rejection_sampling_verify_06_amd import _lib
    return _lib, _lib.load()


def test_destroy_null_and_run_without_context():
    _lib, lib = _lib_loaded()
    lib.spec_verify_destroy(None)                       # NULL is accepted
    a = _lib.SpecVerifyArgs()
    assert lib.spec_verify_run(None, ctypes.byref(a), None) == _lib.SV_ERR_INVALID
    assert b"NULL" in lib.spec_verify_last_error()
    assert lib.spec_verify_run(None, None, None) == _lib.SV_ERR_INVALID
    assert lib.spec_verify_timing_enable(None, 4) == _lib.SV_ERR_INVALID
    calls = ctypes.c_int32()
    ms = (ctypes.c_double * _lib.SV_NUM_KERNELS)()
    assert lib.spec_verify_timing_read(None, ctypes.byref(calls), ms) == _lib.SV_ERR_INVALID


@pytest.mark.parametrize("max_batch,max_k,max_vocab", [(0, 8, 1000), (4097, 8, 1000), (4, 0, 1000), (4, 129, 1000),
                                                        (4, 8, 0), (4, 8, 2097153)])
def test_create_rejects_bad_sizes(max_batch, max_k, max_vocab):
    _lib, lib = _lib_loaded()
    h = ctypes.c_void_p(12345)
    assert lib.spec_verify_create(ctypes.byref(h), 0, max_batch, max_k, max_vocab) == _lib.SV_ERR_INVALID
    assert h.value is None                              # *out is cleared on failure
    assert lib.spec_verify_last_error()
    assert lib.spec_verify_create(None, 0, 4, 8, 1000) == _lib.SV_ERR_INVALID


def test_side_entry_points_reject_bad_arguments():
    _lib, lib = _lib_loaded()
    assert lib.spec_verify_ngram_propose(None, None) == _lib.SV_ERR_INVALID
    g = _lib.SpecVerifyNgramArgs()
    g.batch, g.min_n, g.max_n, g.max_tokens = 2, 3, 2, 5       # min_n > max_n
    assert lib.spec_verify_ngram_propose(ctypes.byref(g), None) == _lib.SV_ERR_INVALID
    g.min_n, g.max_n, g.max_tokens = 1, 17, 5                   # window past the limit
    assert lib.spec_verify_ngram_propose(ctypes.byref(g), None) == _lib.SV_ERR_INVALID
    g.max_n, g.max_tokens = 4, 129
    assert lib.spec_verify_ngram_propose(ctypes.byref(g), None) == _lib.SV_ERR_INVALID
    assert lib.spec_verify_stats_accumulate(4, 0, None, None, None, None) == _lib.SV_ERR_INVALID
    assert lib.spec_verify_stats_accumulate(4, 8, None, None, None, None) == _lib.SV_ERR_INVALID
    assert lib.spec_verify_stats_summary(129, None, None, None) == _lib.SV_ERR_INVALID
    ad = _lib.SpecVerifyAdaptArgs()
    ad.batch, ad.kind, ad.min_k, ad.max_k, ad.window, ad.min_samples, ad.target, ad.rate = 0, 0, 1, 5, 10, 1, 0.7, 0.1
    ad.count = 2                                                # unknown count
    assert lib.spec_verify_adapt(ctypes.byref(ad), None) == _lib.SV_ERR_INVALID
    assert b"count" in lib.spec_verify_last_error()
    ad.count, ad.kind = 0, 3                                    # unknown kind
    assert lib.spec_verify_adapt(ctypes.byref(ad), None) == _lib.SV_ERR_INVALID
    ad.kind, ad.target = 0, 1.5
    assert lib.spec_verify_adapt_reset(ctypes.byref(ad), 5, None) == _lib.SV_ERR_INVALID
    ad.target = 0.7
    assert lib.spec_verify_adapt_reset(ctypes.byref(ad), 0, None) == _lib.SV_ERR_INVALID   # init_k
    assert lib.spec_verify_adapt(ctypes.byref(ad), None) == _lib.SV_OK                     # batch 0: nothing to do


def test_token_logprobs_rejects_bad_arguments():
    _lib, lib = _lib_loaded()
    ws = lib.spec_verify_logprobs_workspace
    assert 0 < ws(4, 1000, _lib.SV_BF16, 0) < ws(4, 1000, _lib.SV_BF16, 5) < ws(8, 1000, _lib.SV_BF16, 5)
    assert ws(0, 1000, _lib.SV_BF16, 5) == 0
    for rows, vocab, dtype, top in [(-1, 10, 0, 0), (4, 0, 0, 0), (4, 2097153, 0, 0), (4, 10, 2, 0), (4, 10, 0, -1),
                                    (4, 10, 0, 11), (4, 1000, 0, 65), (1 << 31, 10, 0, 0), (1 << 62, 10, 0, 0)]:
        assert ws(rows, vocab, dtype, top) == _lib.SV_ERR_INVALID
    call = lib.spec_verify_token_logprobs
    assert call(None, None) == _lib.SV_ERR_INVALID
    a = _lib.SpecVerifyLogprobsArgs(rows=0, vocab=100, dtype=0, top=0)
    assert call(ctypes.byref(a), None) == _lib.SV_OK                     # no rows: nothing to do
    good = dict(rows=2, vocab=100, dtype=0, top=2, logits=0x1000, ld=100, tokens=0x1000, logprob=0x1000, top_tokens=0x1000,
                workspace=0x1000, workspace_bytes=10000)
    for bad in (dict(logits=None), dict(logits=0x1001), dict(ld=99), dict(ld=1 << 61), dict(tokens=None),
                dict(top_tokens=None), dict(top=0), dict(workspace=None), dict(workspace=0x1008), dict(workspace_bytes=10),
                dict(rows=-1), dict(dtype=3)):
        a = _lib.SpecVerifyLogprobsArgs(**{**good, **bad})
        assert call(ctypes.byref(a), None) == _lib.SV_ERR_INVALID, bad
        assert b"spec_verify_token_logprobs" in lib.spec_verify_last_error(), bad


def test_paged_attention_rejects_bad_arguments():
    _lib, lib = _lib_loaded()
    call, ws = lib.spec_verify_paged_attention, lib.spec_verify_attention_workspace
    assert call(None, None) == ws(None) == _lib.SV_ERR_INVALID
    good = dict(batch=2, total_rows=6, heads=8, kv_heads=2, head_dim=128, dtype=_lib.SV_BF16, page_size=16, num_pages=10, slots=2,
                max_pages=4, page_table_stride=4, q=0x1000, q_row_stride=1024, q_head_stride=128, k=0x1000, k_page_stride=4096,
                k_head_stride=2048, k_token_stride=128, v=0x1000, v_page_stride=4096, v_head_stride=2048, v_token_stride=128,
                page_table=0x1000, seq_len=0x1000, num_draft=0x1000, scale=0.1, out=0x1000, workspace=0x1000,
                workspace_bytes=1 << 30)
    a = _lib.SpecVerifyAttentionArgs(**good)
    assert ws(ctypes.byref(a)) > 0
    sizes = [dict(batch=-1), dict(batch=4097, total_rows=5000), dict(total_rows=1), dict(total_rows=524289), dict(heads=7),
             dict(kv_heads=0), dict(heads=0), dict(heads=514, kv_heads=2), dict(head_dim=96), dict(dtype=_lib.SV_F32), dict(page_size=8),
             dict(page_size=48), dict(page_size=2048), dict(num_pages=0), dict(num_pages=1 << 31), dict(slots=0),
             dict(max_pages=0), dict(max_pages=1 << 30), dict(window=-1),
             dict(batch=4096, total_rows=500000, heads=256, kv_heads=256, max_pages=60000)]
    for bad in sizes:
        a = _lib.SpecVerifyAttentionArgs(**{**good, **bad})
        assert ws(ctypes.byref(a)) == _lib.SV_ERR_INVALID, bad
    for bad in sizes + [dict(q=None), dict(k=None), dict(v=None), dict(page_table=None), dict(seq_len=None),
                        dict(num_draft=None), dict(out=None), dict(q=0x1008), dict(k=0x1002), dict(v=0x1004), dict(out=0x1008),
                        dict(q_row_stride=1020), dict(q_head_stride=-8), dict(k_page_stride=4), dict(k_token_stride=1 << 25),
                        dict(v_head_stride=1), dict(v_token_stride=12), dict(page_table_stride=3), dict(scale=float("nan")),
                        dict(scale=float("inf")), dict(workspace=None), dict(workspace=0x1001), dict(workspace_bytes=100)]:
        a = _lib.SpecVerifyAttentionArgs(**{**good, **bad})
        assert call(ctypes.byref(a), None) == _lib.SV_ERR_INVALID, bad
        assert b"spec_verify_" in lib.spec_verify_last_error()
    a = _lib.SpecVerifyAttentionArgs(**{**good, "batch": 0, "total_rows": 0})
    assert call(ctypes.byref(a), None) == _lib.SV_OK                     # no sequences: nothing to do


def test_cache_rejects_bad_arguments():
    _lib, lib = _lib_loaded()
    good = dict(slots=4, max_pages=8, page_size=16, num_pages=20, layers=2, kv_heads=2, head_dim=64, page_table=0x1000,
                seq_len=0x1000, refcount=0x1000, k=0x1000, v=0x1000, workspace=0x1000, workspace_bytes=1 << 20)
    P = 0x1000

    def every(c):
        r = ctypes.byref(c)
        return [lib.spec_verify_cache_reserve(r, 2, P, P, 3, P, P, P, None), lib.spec_verify_cache_truncate(r, 2, P, P, P, None),
                lib.spec_verify_cache_commit(r, 2, P, P, P, P, None), lib.spec_verify_cache_fork(r, 2, P, P, P, None),
                lib.spec_verify_cache_compact(r, P, None), lib.spec_verify_cache_write(r, 0, 1, P, 128, 64, P, 128, 64, P, None)]
    sizes = [dict(slots=0), dict(slots=4097), dict(max_pages=0), dict(max_pages=131073), dict(page_size=8), dict(page_size=17),
             dict(page_size=2048), dict(num_pages=0), dict(num_pages=1 << 30), dict(layers=0), dict(layers=4097), dict(kv_heads=0),
             dict(head_dim=0), dict(head_dim=12), dict(kv_heads=1024, head_dim=128)]
    for bad in sizes:
        c = _lib.SpecVerifyCache(**{**good, **bad})
        assert lib.spec_verify_cache_workspace(ctypes.byref(c)) == _lib.SV_ERR_INVALID, bad
    for bad in sizes + [dict(page_table=None), dict(seq_len=None), dict(refcount=None), dict(refcount=0x1004), dict(k=None), dict(v=None),
                        dict(k=0x1008), dict(v=0x1002), dict(workspace=None), dict(workspace=0x1008), dict(workspace_bytes=64)]:
        assert every(_lib.SpecVerifyCache(**{**good, **bad})) == [_lib.SV_ERR_INVALID] * 6, bad
    c = _lib.SpecVerifyCache(**good)
    r = ctypes.byref(c)
    assert lib.spec_verify_cache_workspace(r) > 0
    assert lib.spec_verify_cache_workspace(None) == _lib.SV_ERR_INVALID
    INV, OK = _lib.SV_ERR_INVALID, _lib.SV_OK
    for batch in (-1, 5):
        assert lib.spec_verify_cache_reserve(r, batch, P, P, 3, P, P, P, None) == INV
        assert lib.spec_verify_cache_truncate(r, batch, P, P, P, None) == INV
        assert lib.spec_verify_cache_commit(r, batch, P, P, P, P, None) == INV
        assert lib.spec_verify_cache_fork(r, batch, P, P, P, None) == INV
    for num_new, total, start, slots in ((None, 3, P, P), (P, -1, P, P), (P, 524289, P, P), (P, 3, None, P), (P, 3, P, None)):
        assert lib.spec_verify_cache_reserve(r, 2, P, num_new, total, start, slots, P, None) == INV
    assert lib.spec_verify_cache_commit(r, 2, P, None, P, P, None) == INV
    assert lib.spec_verify_cache_commit(r, 2, P, P, None, P, None) == INV
    assert lib.spec_verify_cache_fork(r, 2, None, P, P, None) == INV
    assert lib.spec_verify_cache_fork(r, 2, P, None, P, None) == INV
    for a in ((-1, 1, P, 128, 64, P, 128, 64, P), (2, 1, P, 128, 64, P, 128, 64, P), (0, -1, P, 128, 64, P, 128, 64, P),
              (0, 524289, P, 128, 64, P, 128, 64, P), (0, 1, None, 128, 64, P, 128, 64, P), (0, 1, P, 128, 64, None, 128, 64, P),
              (0, 1, P, 128, 64, P, 128, 64, None), (0, 1, 0x1008, 128, 64, P, 128, 64, P), (0, 1, P, 127, 64, P, 128, 64, P),
              (0, 1, P, 128, 64, P, 128, -64, P)):
        assert lib.spec_verify_cache_write(r, *a, None) == INV, a
        assert b"spec_verify_cache_write" in lib.spec_verify_last_error()
    assert lib.spec_verify_cache_write(r, 0, 0, None, 0, 0, None, 0, 0, None, None) == OK
    assert lib.spec_verify_cache_reserve(r, 0, None, None, 0, None, None, None, None) == OK
    assert lib.spec_verify_cache_fork(r, 0, None, None, None, None) == OK


@pytest.mark.parametrize("scale", [1e39, -1e39, 3e38])
def test_paged_attention_rejects_a_scale_outside_32_bits(scale):
    """The scores are float32: a scale (times log2 e) that is infinite there
    would turn a score of 0 into NaN."""
    _lib, lib = _lib_loaded()
    a = _lib.SpecVerifyAttentionArgs(
        batch=2, total_rows=6, heads=8, kv_heads=2, head_dim=128, dtype=_lib.SV_BF16, page_size=16, num_pages=10, slots=2,
        max_pages=4, page_table_stride=4, q=0x1000, q_row_stride=1024, q_head_stride=128, k=0x1000, k_page_stride=4096,
        k_head_stride=2048, k_token_stride=128, v=0x1000, v_page_stride=4096, v_head_stride=2048, v_token_stride=128,
        page_table=0x1000, seq_len=0x1000, num_draft=0x1000, scale=scale, out=0x1000, workspace=0x1000,
        workspace_bytes=1 << 30)
    assert lib.spec_verify_paged_attention(ctypes.byref(a), None) == _lib.SV_ERR_INVALID
    assert b"scale" in lib.spec_verify_last_error()


def test_paged_attention_rejects_rows_without_a_sequence():
    """No sequences, but rows: the outputs would be left as they were."""
    _lib, lib = _lib_loaded()
    good = dict(batch=0, total_rows=0, heads=8, kv_heads=2, head_dim=128, dtype=_lib.SV_BF16, page_size=16, num_pages=10, slots=2,
                max_pages=4)
    for rows, want in ((0, _lib.SV_OK), (1, _lib.SV_ERR_INVALID), (3, _lib.SV_ERR_INVALID)):
        a = _lib.SpecVerifyAttentionArgs(**{**good, "total_rows": rows})
        assert lib.spec_verify_paged_attention(ctypes.byref(a), None) == want
        assert (lib.spec_verify_attention_workspace(ctypes.byref(a)) < 0) == (want != _lib.SV_OK)


def test_commit_reserved_rejects_bad_arguments():
    _lib, lib = _lib_loaded()
    good = dict(slots=4, max_pages=8, page_size=16, num_pages=20, layers=2, kv_heads=2, head_dim=64, page_table=0x1000,
                seq_len=0x1000, refcount=0x1000, k=0x1000, v=0x1000, workspace=0x1000, workspace_bytes=1 << 20)
    P, call, r = 0x1000, lib.spec_verify_cache_commit_reserved, ctypes.byref(_lib.SpecVerifyCache(**good))
    for a in ((None, 2, P, P, P, P, P), (r, -1, P, P, P, P, P), (r, 5, P, P, P, P, P), (r, 2, P, None, P, P, P),
              (r, 2, P, P, None, P, P), (r, 2, P, P, P, None, P),
              (ctypes.byref(_lib.SpecVerifyCache(**{**good, "workspace": None})), 2, P, P, P, P, P)):
        assert call(*a, None) == _lib.SV_ERR_INVALID, a
        assert b"spec_verify_cache_commit_reserved" in lib.spec_verify_last_error()
    assert call(r, 0, None, None, None, None, None, None) == _lib.SV_OK
