"""Shared prefixes and what is not a number, where a row's part of the work (128
keys or more) holds nothing else: as without groups, the rows that see it are NaN."""
import pytest
import torch

from . import coded_util as cu
from . import serving_util as su
from .test_gpu_attention_shared import KINDS, _call, _i32, _near, _q, sv  # noqa: F401

pytestmark = pytest.mark.gpu

# few rows of a key head go with the sequences' own, more than 48 have tiles of 128 for themselves
FEW = ([(2000, [50] * 4), (300, [400, 7])], [0, 0, 2, 0, 1, 0])
MANY = ([(1500, [50, 400] + [9] * 25), (300, [400, 7])], [i % 3 for i in range(29)])


def _check(sv, made, nd, q, ref, dtype, gone):
    """NaN where ``gone`` ([rows, heads]) says so, with groups and without; else near the reference."""
    o = _call(sv, q, made, nd)
    plain = _call(sv, q, made, nd, groups=None, prefix_len=None)
    for x in (o, plain):
        out, lse = x["out"].cpu(), x["lse"].cpu()
        assert not x["status"].any()
        assert torch.isnan(out[gone]).all() and torch.isnan(lse[gone]).all()
        out[gone], lse[gone] = ref[0].to(dtype)[gone], ref[1].float()[gone]
        _near({"out": out, "lse": lse}, ref, dtype)


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_queries(sv, shape, D, quant, dtype):  # noqa: F811
    groups, nd = shape
    made = cu.make_shared(groups, 16, 2, D, dtype, quant, 41)
    N = sum(nd) + len(nd)
    q = _q(N, 8, D, dtype, 41)
    ref = su.attention_ref(q, *made[1], made[2], made[3], _i32(nd))
    gone = torch.zeros(N, 8, dtype=torch.bool)
    gone[0, 0] = gone[2, 5] = gone[N // 2, 3] = gone[N - 1] = True
    q[gone.cuda()] = torch.nan
    _check(sv, made, nd, q, ref, dtype, gone)


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_runs_of_keys(sv, shape, D, quant, dtype):  # noqa: F811
    """128 and 640 keys of the first group's prefix, then 128 of a sequence's own."""
    groups, nd = shape
    made = cu.make_shared(groups, 16, 2, D, dtype, quant, 42)
    N, first = sum(nd) + len(nd), sum(n + 1 for n in nd[:len(groups[0][1])])
    q = _q(N, 8, D, dtype, 42)
    ref = su.attention_ref(q, *made[1], made[2], made[3], _i32(nd))
    b = len(groups[0][1])                                                    # the sequence of 300 + 400
    for seq, start, count, rows in ((0, 256, 128, slice(0, first)), (0, 512, 640, slice(0, first)), (b, 384, 128, slice(first, first + nd[b] + 1))):
        for what in ("scale", "code") if quant == cu.E4M3 else ("scale",):
            pools = [None if x is None else x.clone() for x in made[0]]
            pages = made[2][seq, start // 16:(start + count) // 16].long()
            if quant is None:
                pools[0][pages] = torch.nan
            elif what == "scale":
                pools[1][pages] = torch.nan
            else:
                pools[0].view(torch.uint8)[pages] = 0x7F
            gone = torch.zeros(N, 8, dtype=torch.bool)
            gone[rows] = True
            _check(sv, (pools, *made[1:]), nd, q, ref, dtype, gone)


@pytest.mark.parametrize("quant,dtype", [x for x in KINDS if x[0] is not None])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_values_of_weight_0(sv, shape, D, quant, dtype):  # noqa: F811
    """128 keys with scores of -inf, for all rows, in front of value scales that are NaN: rows that see them are NaN, their lse is not."""
    groups, nd = shape
    made = cu.make_shared(groups, 16, 2, D, dtype, quant, 43)
    N, first = sum(nd) + len(nd), sum(n + 1 for n in nd[:len(groups[0][1])])
    q = _q(N, 8, D, dtype, 43)
    q[:, :, 0] = -8.0
    b = len(groups[0][1])
    for seq, start, rows in ((0, 256, slice(0, first)), (b, 384, slice(first, first + nd[b] + 1))):
        pools, ref = [x.clone() for x in made[0]], [x.clone() for x in made[1]]
        pages = made[2][seq, start // 16:start // 16 + 8].long()
        codes = pools[0].view(torch.uint8)
        codes[pages] = 0
        codes[pages, :, :, 0] = 0x38 if quant == cu.E4M3 else 1
        pools[1][pages], pools[3][pages] = torch.inf, torch.nan
        ref[0][pages.cpu()] = 0.0
        ref[0][pages.cpu(), :, :, 0] = 1e9                                     # times -8: a weight of 0
        want = su.attention_ref(q, *ref, made[2], made[3], _i32(nd))
        for kw in ({}, dict(groups=None, prefix_len=None)):
            o = _call(sv, q, (pools, *made[1:]), nd, **kw)
            out, lse = o["out"].cpu(), o["lse"].cpu()
            assert torch.isnan(out[rows]).all() and not o["status"].any()
            out[rows] = want[0].to(dtype)[rows]
            _near({"out": out, "lse": lse}, want, dtype)
