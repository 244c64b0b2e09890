"""8-bit pages: codes and scales that are no numbers make the rows that see them
NaN whatever their weight, also in a tile with keys that some rows do not see."""
import pytest
import torch

from . import coded_util as cu
from . import serving_util as su
from .test_gpu_attention_codes import KINDS, _call, _i32, _near, _q, sv  # noqa: F401

pytestmark = pytest.mark.gpu

L, ND, P = [150, 77], [4, 2], 16
AT = [147, 75]                                   # behind it lie keys that some rows do not see
SEE, KEEP = [2, 3, 4, 6, 7], [0, 1, 5]           # the rows that see it, and those that do not


def _made(D, dtype, quant, heads):
    """Pools in which the key at AT has one number: 1 by its code, along a query number of at least 8."""
    pools, ref, table, seq_len = cu.make_coded_pages(L, P, 2, D, dtype, quant, 61)
    q = _q(8, heads, D, dtype, 61)
    q[:, :, 0] = torch.where(q[:, :, 0] < 0, -8.0, 8.0)
    places = [(table[b, n // P].long(), n % P) for b, n in enumerate(AT)]
    for page, off in places:
        codes = pools[0].view(torch.uint8)
        codes[page, :, off] = 0
        codes[page, :, off, 0] = 0x38 if quant == cu.E4M3 else 1
    return pools, ref, table, seq_len, q, places


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,heads", [(64, 4), (64, 16), (128, 4), (128, 16), (256, 8)])
@pytest.mark.parametrize("why", ["weight", "scale"])
def test_a_code_without_a_number_of_weight_0(sv, why, D, heads, dtype):  # noqa: F811
    """Where the key's score is some -2^20 below the others, or the value's scale is 0."""
    pools, ref, table, seq_len, q, places = _made(D, dtype, cu.E4M3, heads)
    q[:, :, 0] = -8.0
    want = su.attention_ref(q, *ref, table, seq_len, _i32(ND))
    for page, off in places:
        pools[1][page, :, off] = 2.0 ** 20
        if why == "scale":
            pools[1][page, :, off], pools[3][page, :, off] = 2.0 ** -10, 0.0
        pools[2].view(torch.uint8)[page, :, off, 5] = 0x7F
        pools[2].view(torch.uint8)[page, :, off, D - 1] = 0xFF
    o = _call(sv, q, pools, table, seq_len, ND)
    assert torch.isnan(o["out"][SEE][..., [5, D - 1]]).all()
    assert torch.isfinite(o["out"][SEE][..., 6:D - 1]).all() and torch.isfinite(o["lse"]).all()
    _near(o, want, dtype, KEEP)


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D,heads", [(64, 4), (64, 16), (128, 4), (128, 16), (256, 8)])
@pytest.mark.parametrize("x", [torch.nan, torch.inf, -torch.inf])
def test_a_value_scale_that_is_not_finite(sv, x, D, heads, quant, dtype):  # noqa: F811
    """Next to weights of their own, of 0 (by underflow), and of a score of -inf."""
    for key_scale in (2.0 ** -10, 2.0 ** 20, torch.inf):
        pools, ref, table, seq_len, q, places = _made(D, dtype, quant, heads)
        q[:, :, 0] = -8.0
        want = su.attention_ref(q, *ref, table, seq_len, _i32(ND))
        for page, off in places:
            pools[1][page, :, off], pools[3][page, :, off] = key_scale, x
        o = _call(sv, q, pools, table, seq_len, ND)
        assert not torch.isfinite(o["out"][SEE]).any() and torch.isfinite(o["lse"]).all()
        _near(o, want, dtype, KEEP)


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_key_scale_that_is_infinite(sv, D, quant, dtype):  # noqa: F811
    """Scores of -inf have no weight, those of +inf leave a row without a number."""
    pools, ref, table, seq_len, q, places = _made(D, dtype, quant, 8)
    for page, off in places:
        pools[1][page, :, off] = torch.inf
        ref[0][page, :, off] = 0.0
        ref[0][page, :, off, 0] = 1e6
    want = su.attention_ref(q, *ref, table, seq_len, _i32(ND))
    o = _call(sv, q, pools, table, seq_len, ND)
    gone = torch.zeros(8, 8, dtype=torch.bool)
    gone[SEE] = q[SEE][:, :, 0].cpu() > 0
    assert gone[SEE].any() and not gone[SEE].all()
    out, lse = o["out"].cpu(), o["lse"].cpu()
    assert torch.isnan(out[gone]).all() and torch.isnan(lse[gone]).all()
    out[gone] = want[0][gone] = 0
    lse[gone] = want[1][gone] = 0
    _near({"out": out, "lse": lse}, want, dtype)
