"""How many bits of a softmax weight reach the attention's second product,
against closed forms in float64.

Outputs are rounded once: off by at most U = finfo.eps / 2 relative (bfloat16
2^-8, float16 2^-11)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_06_amd as m
    return m


@pytest.mark.parametrize("D,H", [(64, 4), (64, 24), (64, 64), (128, 4), (128, 24), (128, 40), (128, 64), (256, 4), (256, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_weight_keeps_the_bits_of_float32(sv, D, H, dtype):
    """Two keys whose weighted values nearly cancel, so that the output is
    2^-11 of its terms and shows a weight's last bits.  Weights 1 and p, p from
    0.3 to 0.8; values -2 and x = 2 / p: out = (x p - 2) / (1 + p).

    The score, |s| < 2 in log2 units, is off by 2^-24 from its own rounding, as
    much from the constant's, and twice 2^-24 * 1.45 from the product's: p by
    5 * 2^-24 ln 2 relative, by 2^-23 more from the exponential.  Its two 16-bit
    halves are off by half a step twice: 2^-16 for bfloat16, 2^-22 for float16.
    With x p = 2 and 1 + p > 1.3 the output is off by less than 2^-15 and 2^-20
    in front of its own rounding; one half alone would be off by up to 2^-7 and
    2^-10."""
    B = 60
    g = torch.Generator().manual_seed(D + H)
    k, v = torch.zeros(B, 1, 16, D, dtype=dtype), torch.zeros(B, 1, 16, D, dtype=dtype)
    x = torch.tensor([2.5, 3.5, 4.5, 5.5, 6.5], dtype=torch.float64).repeat(B // 5)
    s = torch.log(2 / x) + (torch.rand(B, generator=g, dtype=torch.float64) - 0.5) * 2.0 ** -11
    for d in range(3):                                    # the score in three parts, each exact in the type
        k[:, 0, 1, d] = s.to(dtype)
        s = s - k[:, 0, 1, d].double()
    v[:, 0, 0], v[:, 0, 1] = -2.0, x.to(dtype)[:, None]
    q = torch.zeros(B, H, D, dtype=dtype)
    q[:, :, 0] = 1.0
    q[:, :, 1] = 1.0
    q[:, :, 2] = 1.0 + torch.arange(H) / 64.0             # every head its own last bits
    s = (q.double() * k[:, :, 1].double()).sum(-1)
    want = (x[:, None] * s.exp() - 2) / (1 + s.exp())
    assert want.abs().max() < 2.0 ** -7
    i32 = dict(dtype=torch.int32, device="cuda")
    o = sv.paged_attention(q.cuda(), k.cuda(), v.cuda(), torch.arange(B, **i32)[:, None], torch.full((B,), 2, **i32),
                           torch.zeros(B, **i32), scale=1.0)
    got = o["out"].cpu().double()
    off = (got - want[:, :, None]).abs() - U[dtype] * want.abs()[:, :, None]
    assert off.max() < {torch.bfloat16: 2.0 ** -15, torch.float16: 2.0 ** -20}[dtype], math.log2(off.max())


@pytest.mark.parametrize("gap", [13.0, 14.5, 16.0, 17.375, 20.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,H,B,L,at", [(128, 8, 32, 4097, 0), (128, 24, 64, 1025, 0), (64, 128, 64, 1025, 0), (64, 8, 128, 1025, 700),
                                        (256, 8, 32, 1025, 0)])
def test_a_flat_tail_far_below_a_sink(sv, D, H, B, L, at, dtype, gap):
    """One key whose value is 0, `gap` nats above all others, whose values are
    64: the output is the others' share alone.  As many (sequence, key head)
    tiles as blocks, so that a wave holds a quarter of the keys against the
    sink; the other waves' weights are large and scaled in float32.

    The scores are exact but for 2^-20 (the product with log2 e, up to 28.9)
    and 2^-20 (the constant): weights by 2^-19.5 relative.  Sums of L / 128
    vectors of 8 in order: L / 16 * 2^-24.  A weight's float16 halves are held
    to half a step of 2^-38, 2^-39 of the sink's, which is 2^-10 of a weight 20
    nats below and applies to a quarter of them: 2^-12 (bfloat16 2^-16).  Then
    the output's own rounding: 1/16 more of it is more than all of that but the
    2^-12, which gets its own."""
    i32 = dict(dtype=torch.int32, device="cuda")
    KV, per = 8, -(-L // 16)
    k = torch.zeros(B * per, KV, 16, D, dtype=dtype, device="cuda")
    v = torch.full_like(k, 64.0)
    table = torch.arange(B * per, **i32).view(B, per)
    sink = table[:, at // 16].long()
    k[sink, :, at % 16, 0] = gap
    v[sink, :, at % 16] = 0.0
    q = torch.zeros(B, H, D, dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    o = sv.paged_attention(q, k, v, table, torch.full((B,), L, **i32), torch.zeros(B, **i32), scale=1.0, want_lse=True)
    tail = (L - 1) * math.exp(-gap)
    want = 64 * tail / (1 + tail)
    assert want > 2.0 ** -14                                # a normal number of the type
    got = o["out"].cpu().double()
    assert (got - want).abs().max() <= want * (U[dtype] * 17 / 16 + 2.0 ** -12), ((got - want).abs().max() / want).item()
    # lse: in log2 units 2^-20 from the score's product, 2^-19.7 from the constant, 2^-20 from M + log2 L and 2^-21 from
    # log2 L, in nats 2^-20 from the result's rounding and 2^-20.7 from ln 2: 4.0e-6 < 2^-17 for a score up to 28.9.
    # L itself: the lane that holds the sink adds L / 16 weights to a sum near the sink's (1 / 4 of the keys go to its
    # wave, 1 / 4 of those to it), and each addition is off by up to half a step there, 2^-24 of it, to the same side.
    assert (o["lse"].cpu().double() - (gap + math.log1p(tail))).abs().max() < 2.0 ** -17 + L / 16 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", [2.0 ** 22, 2.0 ** 24, 2.0 ** 26, 2.0 ** 28])
def test_scores_of_any_size(sv, dtype, size):
    """Scores around +-size log2 units, in steps far above what a float32 holds
    there: the largest key takes all, whatever the weights are taken against."""
    g = torch.Generator().manual_seed(int(math.log2(size)))
    L, B, D = 700, 6, 64
    per = -(-L // 16)
    k = torch.zeros(B * per, 1, 16, D)
    step = torch.randint(-64, 65, (B, per * 16), generator=g).float()
    k[:, 0, :, 0] = step.view(-1, 16)
    v = torch.randn(B * per, 1, 16, D, generator=g).to(dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(B * per, **i32).view(B, per)
    q = torch.zeros(B, 2, D)
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    scale = size / 64 * math.log(2)
    o = sv.paged_attention(q.to(dtype).cuda(), k.to(dtype).cuda(), v.cuda(), table, torch.full((B,), L, **i32), torch.zeros(B, **i32),
                           scale=scale, want_lse=True)
    for b in range(B):
        x, vv = step[b, :L].double(), v.view(B, per * 16, D)[b, :L].double()
        for h, sign in enumerate((1.0, -1.0)):
            best = (x * sign) == (x * sign).max()
            want = vv[best].mean(0)
            got = o["out"][b, h].cpu().double()
            assert ((got - want).abs() <= U[dtype] * want.abs() + 2.0 ** -15).all(), (b, h)
            top = (x * sign).max().item() * scale
            assert abs(o["lse"][b, h].item() - top) <= abs(top) * 2.0 ** -22 + math.log(best.sum().item()) + 1e-3


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_sum_over_a_long_row(sv, dtype):
    """131072 keys 17.4 nats below a sink that their block reads first: one at
    a time each is less than half a step of the sum next to it.

    The sink's lane holds 1/16 of the keys and adds them up in eights, L / 128
    additions to a sum near the sink's weight, each off by half a step, 2^-24
    of it.  The rest, 2^-17, is as in the test above."""
    i32 = dict(dtype=torch.int32, device="cuda")
    KV, B, D, P, L, gap = 8, 32, 128, 1024, 131073, 17.375
    per = -(-L // P)
    k = torch.zeros(per, KV, P, D, dtype=dtype, device="cuda")
    v = torch.full_like(k, 64.0)
    k[0, :, 0, 0] = gap
    v[0, :, 0] = 0.0
    table = torch.arange(per, **i32).repeat(B, 1)           # every sequence the same pages
    q = torch.zeros(B, KV, D, dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    o = sv.paged_attention(q, k, v, table, torch.full((B,), L, **i32), torch.zeros(B, **i32), scale=1.0, want_lse=True)
    tail = (L - 1) * math.exp(-gap)
    assert (o["lse"].cpu().double() - (gap + math.log1p(tail))).abs().max() < 2.0 ** -17 + L / 128 * 2.0 ** -24
    want = 64 * tail / (1 + tail)
    assert (o["out"].cpu().double() - want).abs().max() <= want * (U[dtype] * 17 / 16 + 2.0 ** -12)
