"""A captured write of rotated keys and values, replayed with other contents: every place, scale and query it writes."""
import pytest
import torch

from . import coded_util as cu
from .test_gpu_rope import _cache, _case, _cuda, _i32, _parts, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant", [None, cu.E4M3, cu.INT8])
def test_every_place_of_a_replayed_write(sv, quant):  # noqa: F811
    H, KV, D, rows = 4, 2, 128, 37
    qkv, pos, f, w = _case(rows, H, KV, D, D, torch.bfloat16, 7, True)
    dev, p, fd, wq, wk = _cuda(qkv, pos, f, *w)
    q, k, v = _parts(dev, H, KV)
    c = _cache(sv, quant, KV, D, torch.bfloat16)
    held = [x for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None]
    for x in held:
        x.view(torch.uint8).fill_(0x5A)
    r = c.reserve(None, _i32([rows]), rows)
    page, off = r["slots"] // c.page_size, r["slots"] % c.page_size
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = c.write_rotated(1, q, k, v, r["slots"], p, fd, q_weight=wq, k_weight=wk)
    for seed in (8, 9, 10, 11):
        qkv, pos, _, _ = _case(rows, H, KV, D, D, torch.bfloat16, seed, True)
        dev.copy_(qkv), p.copy_(pos)
        g.replay()
        torch.cuda.synchronize()
        before = [x[0].clone() for x in held]
        eager = c.write_rotated(0, q, k, v, r["slots"], p, fd, q_weight=wq, k_weight=wk)
        assert torch.equal(eager, got)
        for x, old in zip(held, before):
            a, b, old = (t.view(torch.uint8) for t in (x[0], x[1], old))
            # the same in both layers, other than it was, and nothing beside it
            n = 4 if x.dtype == torch.float32 else x.element_size() * D
            a, b, old = (t.reshape(*x.shape[1:4], n) for t in (a, b, old))
            assert torch.equal(a[page, :, off], b[page, :, off])
            if x is c.k or x is c.v:
                assert (a[page, :, off] != old[page, :, off]).any(-1).all()
            a = a.clone()
            a[page, :, off] = 0x5A
            b = b.clone()
            b[page, :, off] = 0x5A
            assert (a == 0x5A).all() and (b == 0x5A).all()
