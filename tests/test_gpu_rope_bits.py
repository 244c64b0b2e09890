"""What is neither normed nor rotated goes through unchanged: every 16-bit number,
as a value into the cache, as a key and a query of rotary 0, and read back."""
import pytest
import torch

from .test_gpu_rope import _cache, _i32, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_number(sv, dtype):  # noqa: F811
    D, KV = 128, 8
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).view(-1, KV, D).cuda()
    rows = x.shape[0]
    c = sv.PagedCache(layers=1, num_pages=8, page_size=16, kv_heads=KV, head_dim=D, max_seqs=1, max_pages=8, dtype=dtype, device="cuda")
    r = c.reserve(None, _i32([rows]), rows, want_positions=True)
    f = torch.empty(0, dtype=torch.float64, device="cuda")
    q = c.write_rotated(0, x, x, x, r["slots"], r["positions"], f)
    o = c.read(0, None, _i32([0]), _i32([rows]), rows)
    plain = sv.qk_norm_rope(x, x, r["positions"], f)
    finite = ~torch.isnan(x)
    for got in (q, o["k"], o["v"], plain["q"], plain["k"]):
        assert torch.equal(got.view(torch.int16)[finite], x.view(torch.int16)[finite]) and torch.isnan(got[~finite]).all()


def test_no_rows(sv):  # noqa: F811
    c = _cache(sv, None, 2, 64, torch.bfloat16)
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    r = c.reserve(None, _i32([0, 0]), 0, want_positions=True)
    assert r["status"].tolist() == [0, 0] and r["positions"].numel() == 0
    q = c.write_rotated(0, none, none[:, :2], none[:, :2], r["slots"], r["positions"], f)
    assert q.shape == none.shape and sv.qk_norm_rope(none, none, r["positions"], f)["k"].shape == none.shape
    o = c.read(0, None, _i32([0, 0]), _i32([0, 0]), 0)
    assert o["status"].tolist() == [0, 0] and o["k"].shape == (0, 2, 64)
    for groups in (None, _i32([0])):
        a = c.attend(0, none, _i32([]), groups=groups, prefix_len=None if groups is None else _i32([]))
        assert a["out"].shape == none.shape and a["status"].numel() == 0
