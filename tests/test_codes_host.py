"""What the host refuses of the 8-bit cache and of norms with rotation, before any HIP call (no device needed)."""
import ctypes

import pytest
import torch

from .test_abi import _lib_loaded


def _cache(_lib, **kw):
    sizes = dict(slots=4, max_pages=8, page_size=16, num_pages=32, layers=2, kv_heads=2, head_dim=64)
    sizes.update({k: v for k, v in kw.items() if k in sizes})
    c = _lib.SpecVerifyCache(**sizes)
    c.page_table, c.seq_len, c.refcount, c.k, c.v, c.workspace = 4096, 4096, 4096, 4096, 4096, 4096
    c.workspace_bytes = 1 << 30
    return c


def _codes(_lib, **kw):
    q = _lib.SpecVerifyCodes(_lib.SV_CODES_E4M3, _lib.SV_BF16, 4096, 4096)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def _ref(x):
    return None if x is None else ctypes.byref(x)


@pytest.mark.parametrize("cache,codes,what", [
    ({}, dict(codes=0), "codes 0"), ({}, dict(codes=3), "codes 3"), ({}, dict(dtype=0), "dtype 0"), ({}, dict(k_scale=None), "k_scale"),
    ({}, dict(v_scale=4100), "v_scale"), (dict(head_dim=24), {}, "head_dim"), (dict(head_dim=528), {}, "head_dim")])
def test_coded_cache_rejects_bad_codes(cache, codes, what):
    _lib, lib = _lib_loaded()
    c, q = _cache(_lib, **cache), _codes(_lib, **codes)
    calls = [lambda: lib.spec_verify_coded_cache_reserve(_ref(c), _ref(q), 1, None, 4096, 1, 4096, 4096, None, None, None),
             lambda: lib.spec_verify_coded_cache_compact(_ref(c), _ref(q), None, None),
             lambda: lib.spec_verify_coded_cache_write(_ref(c), _ref(q), 0, 1, 4096, 128, 64, 4096, 128, 64, 4096, None),
             lambda: lib.spec_verify_cache_read(_ref(c), _ref(q), _lib.SV_BF16, 0, 1, None, 4096, 4096, 1, 4096, 4096, None, None)]
    for f in calls:
        assert f() == _lib.SV_ERR_INVALID
        assert what.encode() in lib.spec_verify_last_error()


def test_coded_write_and_read_reject_bad_arguments():
    _lib, lib = _lib_loaded()
    c, q = _cache(_lib), _codes(_lib)

    def write(codes=q, layer=0, rows=1, k=4096, kr=128, kh=64, v=4096, slots=4096, cache=c):
        return lib.spec_verify_coded_cache_write(_ref(cache), _ref(codes), layer, rows, k, kr, kh, v, 128, 64, slots, None)

    for kw in (dict(codes=None), dict(cache=None), dict(layer=2), dict(layer=-1), dict(rows=-1), dict(rows=524289), dict(k=None), dict(k=4100),
               dict(kr=4), dict(kh=-8), dict(v=None), dict(slots=None), dict(cache=_cache(_lib, kv_heads=2049, head_dim=16))):
        assert write(**kw) == _lib.SV_ERR_INVALID, kw
    assert write(rows=0) == _lib.SV_OK

    def read(codes=q, dtype=_lib.SV_BF16, layer=0, batch=1, first=4096, count=4096, total=1, k=4096, v=4096):
        return lib.spec_verify_cache_read(_ref(c), _ref(codes), dtype, layer, batch, None, first, count, total, k, v, None, None)

    for kw in (dict(dtype=0), dict(dtype=_lib.SV_F16), dict(layer=2), dict(batch=4097), dict(batch=-1), dict(first=None), dict(count=None),
               dict(total=-1), dict(total=524289), dict(k=None), dict(v=4104), dict(batch=0), dict(codes=None, dtype=7)):
        assert read(**kw) == _lib.SV_ERR_INVALID, kw
    assert read(batch=0, total=0) == _lib.SV_OK
    for f, a in ((lib.spec_verify_coded_cache_reserve, (1, None, None, 1, 4096, 4096, None, None, None)),
                 (lib.spec_verify_coded_cache_reserve, (1, None, 4096, -1, 4096, 4096, None, None, None)),
                 (lib.spec_verify_coded_cache_reserve, (9, None, 4096, 1, 4096, 4096, None, None, None))):
        assert f(_ref(c), _ref(q), *a) == _lib.SV_ERR_INVALID
    assert lib.spec_verify_coded_cache_reserve(_ref(c), _ref(q), 0, None, None, 0, None, None, None, None, None) == _lib.SV_OK


def _rope(_lib, **kw):
    a = _lib.SpecVerifyRopeArgs(rows=3, heads=4, kv_heads=2, head_dim=64, rotary=64, dtype=_lib.SV_BF16, eps=1e-6, q=4096, q_row_stride=256,
                                q_head_stride=64, k=4096, k_row_stride=128, k_head_stride=64, positions=4096, inv_freq=4096, q_out=4096, k_out=4096)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_norms_with_rotation_reject_bad_arguments():
    _lib, lib = _lib_loaded()
    for kw in (dict(dtype=0), dict(head_dim=8), dict(head_dim=72), dict(head_dim=528), dict(rotary=8), dict(rotary=80), dict(rotary=-16),
               dict(heads=0), dict(kv_heads=0), dict(heads=4095), dict(rows=-1), dict(rows=524289), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(q=None), dict(k=None), dict(positions=None), dict(inv_freq=None), dict(q_out=None), dict(k_out=None),
               dict(v=4096), dict(slots=4096), dict(q=4100), dict(k_out=4104), dict(q_weight=4104), dict(q_row_stride=4), dict(k_head_stride=-8),
               dict(q_weight=4096, weight_dtype=_lib.SV_F16)):
        assert lib.spec_verify_qk_norm_rope(_ref(_rope(_lib, **kw)), None, None, None) == _lib.SV_ERR_INVALID, kw
    assert lib.spec_verify_qk_norm_rope(None, None, None, None) == _lib.SV_ERR_INVALID
    assert lib.spec_verify_qk_norm_rope(_ref(_rope(_lib, rows=0)), None, None, None) == _lib.SV_OK
    # with a cache
    into = dict(v=4096, v_row_stride=128, v_head_stride=64, slots=4096, k_out=None)
    c, q = _cache(_lib), _codes(_lib)
    for cache, codes, kw in ((c, None, dict(v=None)), (c, None, dict(slots=None)), (c, None, dict(k_out=4096)), (c, None, dict(layer=2)),
                             (c, None, dict(layer=-1)), (c, None, dict(kv_heads=1)), (c, None, dict(head_dim=128)), (c, None, dict(v_row_stride=4)),
                             (c, _codes(_lib, dtype=_lib.SV_F16), {}), (c, _codes(_lib, codes=5), {}), (None, q, dict(v=None, slots=None, k_out=4096))):
        assert lib.spec_verify_qk_norm_rope(_ref(_rope(_lib, **{**into, **kw})), _ref(cache), _ref(codes), None) == _lib.SV_ERR_INVALID, kw
    assert lib.spec_verify_qk_norm_rope(_ref(_rope(_lib, **{**into, "rows": 0})), _ref(c), _ref(q), None) == _lib.SV_OK


def test_python_checks_before_the_library():
    import rejection_sampling_verify_06_amd as sv
    x, f = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        sv.qk_norm_rope(x, x, torch.zeros(2, dtype=torch.int32), f)               # not on a GPU
    with pytest.raises(ValueError):
        sv.qk_norm_rope(x[0], x, torch.zeros(2, dtype=torch.int32), f)
    with pytest.raises(ValueError):
        sv.PagedCache(1, 8, 16, 2, 64, 2, 4, quant="e5m2")


def _attn(_lib, **kw):
    a = _lib.SpecVerifyAttentionArgs(batch=2, total_rows=3, heads=4, kv_heads=2, head_dim=64, dtype=_lib.SV_BF16, page_size=16, window=0, num_pages=32,
                                     slots=2, max_pages=8, page_table_stride=8, q=4096, q_row_stride=256, q_head_stride=64, k=4096, k_page_stride=2048,
                                     k_head_stride=1024, k_token_stride=64, v=4096, v_page_stride=2048, v_head_stride=1024, v_token_stride=64,
                                     page_table=4096, seq_len=4096, num_draft=4096, scale=0.125, out=4096, workspace=4096, workspace_bytes=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _options(_lib, **kw):
    o = _lib.SpecVerifyAttentionOptions(codes=_lib.SV_CODES_INT8, k_scale=4096, k_scale_page_stride=32, k_scale_head_stride=16, v_scale=4096,
                                        v_scale_page_stride=32, v_scale_head_stride=16, num_groups=1, groups=4096, prefix_len=4096)
    for k, v in kw.items():
        setattr(o, k, v)
    return o


def test_attention_options_reject_bad_arguments():
    """All but the workspace is in order, which is asked for last."""
    _lib, lib = _lib_loaded()

    def call(o, **kw):
        a = _attn(_lib, **kw)
        assert lib.spec_verify_paged_attention_options(_ref(a), _ref(o), None) == _lib.SV_ERR_INVALID
        return lib.spec_verify_last_error().decode()

    assert "workspace" in call(_options(_lib)) and "workspace" in call(_options(_lib, codes=0, k_scale=None)) and "workspace" in call(None)
    for o, a, what in ((dict(codes=3), {}, "codes"), (dict(codes=-1), {}, "codes"), (dict(k_scale=None), {}, "k_scale"), (dict(v_scale=4104), {}, "v_scale"),
                       (dict(k_scale_page_stride=30), {}, "scales"), (dict(v_scale_head_stride=-4), {}, "scales"),
                       ({}, dict(k_token_stride=72), "codes"), ({}, dict(v_page_stride=8), "codes"), (dict(num_groups=-1), {}, "num_groups"),
                       (dict(num_groups=3), {}, "num_groups"), ({}, dict(window=5), "window"), (dict(groups=None), {}, "groups"),
                       (dict(prefix_len=None), {}, "prefix_len")):
        assert what in call(_options(_lib, **o), **a), (o, a)
    plain = lib.spec_verify_attention_workspace(_ref(_attn(_lib)))
    assert plain == lib.spec_verify_attention_options_workspace(_ref(_attn(_lib)), None) > 0
    shared = lib.spec_verify_attention_options_workspace(_ref(_attn(_lib)), _ref(_options(_lib)))
    assert shared >= 3 * 4 * (64 + 1) * 4 + 2 * 6 * 4                       # the state alone
    assert lib.spec_verify_attention_options_workspace(_ref(_attn(_lib)), _ref(_options(_lib, num_groups=5))) == _lib.SV_ERR_INVALID
    assert lib.spec_verify_paged_attention_options(_ref(_attn(_lib, batch=0, total_rows=0)), _ref(_options(_lib, num_groups=0)), None) == _lib.SV_OK
