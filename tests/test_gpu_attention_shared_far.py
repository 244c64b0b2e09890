"""Shared prefixes of many rows in pools beyond 2^32 bytes, in pages whose
strides do not fit 32 bits, and as many groups as a call may have."""
import pytest
import torch

from . import coded_util as cu
from . import serving_util as su
from .test_gpu_attention_shared import _call, _i32, _near, _q, sv  # noqa: F401

pytestmark = pytest.mark.gpu

P, D, H = 64, 64, 64                             # one key head: 64 rows for each query


def _made(quant, seed):
    return cu.make_shared([(200, [9, 70]), (64, [1])], P, 1, D, torch.bfloat16, quant, seed, extra=0)


def _compare(sv, made, at, k, ks, v, vs):
    q = _q(5, H, D, torch.bfloat16, 71)
    nd = [1, 1, 0]
    o = _call(sv, q, ([k, ks, v, vs], None, at, *made[3:]), nd)
    plain = _call(sv, q, ([k, ks, v, vs], None, at, *made[3:]), nd, groups=None, prefix_len=None)
    assert not o["status"].any() and not plain["status"].any()
    ref = su.attention_ref(q, *made[1], made[2], made[3], _i32(nd))
    _near(o, ref, torch.bfloat16)
    _near(plain, ref, torch.bfloat16)


@pytest.mark.parametrize("quant", [None, cu.INT8])
@pytest.mark.parametrize("alike", [True, False])
def test_far_pages(sv, alike, quant):  # noqa: F811
    """K and V with the same strides, and V with its own."""
    made = _made(quant, 71)
    few = made[0][0].shape[0]
    es = 2 if quant is None else 1
    n = (1 << 32) // (P * D * es) + few + 5
    far = torch.arange(n - few, n, dtype=torch.int32, device="cuda")
    pools = []
    for i in (0, 2):
        x, scale = made[0][i], made[0][i + 1]
        wide = D if i == 0 or alike else 2 * D
        big = torch.empty(n, 1, P, wide, dtype=torch.int16 if quant is None else torch.int8, device="cuda")[..., :D].view(x.dtype)
        big[far.long()] = x
        s = None
        if scale is not None:
            s = torch.empty(n, 1, P, device="cuda")
            s[far.long()] = scale
        pools += [big, s]
    at = torch.where(made[2] < 0, made[2], far[made[2].clamp(min=0).long()])
    _compare(sv, made, at, *pools)


@pytest.mark.parametrize("quant", [None, cu.E4M3])
def test_page_strides_beyond_32_bits(sv, quant):  # noqa: F811
    """The kernel for many rows takes strides of up to 32 bits: another one serves these."""
    made = _made(quant, 72)
    few = made[0][0].shape[0]
    es = 2 if quant is None else 1
    stride = (1 << 32) // es + 16
    flat = torch.empty((few - 1) * stride + 2 * P * D, dtype=made[0][0].dtype, device="cuda")
    pools = []
    for i in (0, 2):
        big = torch.as_strided(flat, (few, 1, P, D), (stride, P * D, D, 1), i // 2 * P * D)
        for p in range(few):
            big[p].view(torch.int16 if quant is None else torch.int8).copy_(made[0][i][p].view(torch.int16 if quant is None else torch.int8))
        pools += [big, made[0][i + 1]]
    _compare(sv, made, made[2], *pools)


@pytest.mark.parametrize("quant", [None, cu.E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_as_many_groups_as_sequences(sv, D, quant):  # noqa: F811
    """4096 groups of one sequence with 64 rows of a key head each."""
    dtype = torch.bfloat16
    made = cu.make_shared([(40, [1 + i % 5 for i in range(4096)])], 16, 1, D, dtype, quant, 73)
    q, nd = _q(4096, H, D, dtype, 73), [0] * 4096
    want = _call(sv, q, made, nd, groups=None, prefix_len=None)
    o = _call(sv, q, made, nd, groups=_i32(list(range(4097))), prefix_len=_i32([40, 33] * 2048))
    assert not o["status"].any()
    # both are float32 until they are rounded, each by half a step of 2^-8 at most
    assert ((o["out"].double() - want["out"].double()).abs() <= 2.0 ** -7 * want["out"].double().abs() + 1e-4).all()
    assert (o["lse"] - want["lse"]).abs().max() < 1e-5
