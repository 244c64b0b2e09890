"""Scales of 0 (also one that is 0 in 32 bits only, and a subnormal one) and
below 0 in the tiles made for many rows behind a shared prefix that ends inside a tile."""
import pytest
import torch

from . import coded_util as cu
from .test_gpu_attention_shared import KINDS, _call, _q, _run, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, 1e-60, 1e-40, -0.08])
def test_scale(sv, scale, D, quant, dtype):  # noqa: F811
    """Scores of -0.08 q.k have a deviation of 0.6 to 1.3: tolerances as elsewhere."""
    _run(sv, [(1007, [9, 60, 4] * 6), (5, [3, 7, 200])], [i % 4 for i in range(18)] + [1, 0, 3], 8, 2, D, 16, dtype, quant, seed=51, scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scale_of_few_rows(sv, dtype):  # noqa: F811
    """20 to 24 rows of a key head, which have those tiles behind long prefixes."""
    for scale in (0.0, -0.08):
        _run(sv, [(9001, [5, 9, 3]), (8011, [7, 2])], [1, 2, 0, 3, 0], 64, 16, 128, 16, dtype, seed=52, scale=scale)


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("x", [torch.inf, -torch.inf])
def test_scale_0_of_infinite_scores(sv, x, quant, dtype):  # noqa: F811
    """0 times an infinite score is no number, as without groups."""
    made = cu.make_shared([(1007, [9, 60, 4] * 6), (5, [3, 7, 200])], 16, 2, 64, dtype, quant, 53)
    nd = [0] * 21
    q = _q(21, 16, 64, dtype, 53)
    q[:, :, 0] = 1.0
    pools = [None if t is None else t.clone() for t in made[0]]
    page = made[2][0, 20].long()
    if quant is None:
        pools[0][page, :, 5, 0] = x
    else:
        codes = pools[0].view(torch.uint8)
        codes[page, :, 5] = 0
        codes[page, :, 5, 0] = 0x38 if quant == cu.E4M3 else 1
        pools[1][page, :, 5] = x
    for kw in ({}, dict(groups=None, prefix_len=None)):
        o = _call(sv, q, (pools, *made[1:]), nd, scale=0.0, **kw)
        assert not o["status"].any()
        assert torch.isnan(o["out"][:18]).all() and torch.isnan(o["lse"][:18]).all()
        assert torch.isfinite(o["out"][18:]).all() and torch.isfinite(o["lse"][18:]).all()
