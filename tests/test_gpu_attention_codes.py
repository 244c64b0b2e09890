"""Attention over a paged cache of 8-bit codes on the GPU, against float64 over
what the codes and scales stand for.

Tolerances as for the 16-bit cache: codes are exact in the products' type, a
score is a float32 sum of D exact products times one float32 factor (two
roundings more), a weight takes a scale on (one more) and is held to 2^-17 by
two bfloat16; the result is rounded once.  With |q|, |k|, |v| of the same sizes
as there ATOL = 2^-9 covers a quarter of the worst case, RTOL is one unit."""
import pytest
import torch

from . import coded_util as cu
from . import serving_util as su

pytestmark = pytest.mark.gpu

RTOL = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
ATOL = 2.0 ** -9
KINDS = [(cu.E4M3, torch.bfloat16), (cu.INT8, torch.bfloat16), (cu.E4M3, torch.float16), (cu.INT8, torch.float16)]


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_06_amd as m
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _q(N, H, D, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn(N, H, D, generator=g) * std).to(dtype).cuda()


def _near(o, ref, dtype, rows=None):
    out, lse = ref
    got, l = o["out"].cpu().double(), o["lse"].cpu().double()
    if rows is not None:
        got, l, out, lse = got[rows], l[rows], out[rows], lse[rows]
    assert not torch.isnan(got).any()
    d = (got - out).abs() - RTOL[dtype] * out.abs()
    assert d.max() < ATOL, d.max()
    assert torch.equal(torch.isinf(l), torch.isinf(lse))
    fine = ~torch.isinf(lse)
    assert (l - lse).abs()[fine].max() < 2.0 ** -10 if fine.any() else True


def _call(sv, q, pools, table, seq_len, nd, **kw):
    return sv.paged_attention(q, pools[0], pools[2], table, seq_len, _i32(nd), k_scale=pools[1], v_scale=pools[3], want_lse=True, **kw)


def _run(sv, L, nd, H, KV, D, P, dtype, quant, seed=0, std=1.0, **kw):
    pools, ref, table, seq_len = cu.make_coded_pages(L, P, KV, D, dtype, quant, seed)
    q = _q(sum(n + 1 for n in nd), H, D, dtype, seed, std)
    o = _call(sv, q, pools, table, seq_len, nd, **kw)
    torch.cuda.synchronize()
    assert not o["status"].cpu().any()
    _near(o, su.attention_ref(q, *ref, table, seq_len, _i32(nd), kw.get("seqs"), kw.get("scale"), kw.get("window", 0)), dtype)
    return o


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [1, 15, 16, 17, 32, 33, 128, 129, 1000])
def test_one_token(sv, L, D, quant, dtype):
    _run(sv, [L], [0], 8, 2, D, 16, dtype, quant, seed=L)


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("H,KV,D", [(1, 1, 64), (7, 1, 128), (16, 16, 64), (32, 8, 128), (15, 3, 256), (40, 2, 64), (64, 1, 128), (64, 1, 64),
                                    (40, 1, 256)])
def test_head_groups(sv, H, KV, D, quant, dtype):
    _run(sv, [300, 65, 129], [4, 0, 1], H, KV, D, 32, dtype, quant, seed=H)


@pytest.mark.parametrize("quant", [cu.E4M3, cu.INT8])
@pytest.mark.parametrize("nd", [[8, 8, 8], [0, 31, 2], [63, 0, 0], [128, 1, 0]])
def test_ragged_rows(sv, nd, quant):
    _run(sv, [300, 290, 200], nd, 8, 2, 128, 64, torch.bfloat16, quant, seed=sum(nd))


@pytest.mark.parametrize("quant", [cu.E4M3, cu.INT8])
@pytest.mark.parametrize("window", [1, 31, 100, 128, 1000])
def test_window(sv, window, quant):
    _run(sv, [1, 40, 300, 777], [0, 5, 8, 3], 8, 4, 64, 16, torch.bfloat16, quant, seed=window, window=window)


def test_scale_and_sharp_softmax(sv):
    _run(sv, [500, 200], [2, 1], 4, 1, 128, 16, torch.bfloat16, cu.E4M3, seed=1, scale=0.5)
    _run(sv, [500, 200], [2, 1], 4, 1, 128, 16, torch.float16, cu.INT8, seed=2, scale=0.0)
    _run(sv, [500, 200], [2, 1], 4, 1, 64, 16, torch.float16, cu.E4M3, seed=3, std=4.0)


@pytest.mark.parametrize("quant", [cu.E4M3, cu.INT8])
def test_many_parts_and_pages(sv, quant):
    _run(sv, [20011, 3, 1, 9000], [2, 0, 0, 8], 8, 2, 128, 16, torch.bfloat16, quant, seed=5)
    _run(sv, [12345], [3], 4, 1, 256, 1024, torch.float16, quant, seed=7)
    _run(sv, [30000], [0], 2, 1, 64, 64, torch.bfloat16, quant, seed=6)


@pytest.mark.parametrize("quant,dtype", KINDS)
def test_scales_of_every_size(sv, quant, dtype):
    """Keys and values whose vectors differ by orders of magnitude: small
    values keep their digits (the result is compared by its own size)."""
    L, P, D = [90, 33], 16, 128
    pools, ref, table, seq_len = cu.make_coded_pages(L, P, 2, D, dtype, quant, 21)
    f = 2.0 ** torch.randint(-30, -9, pools[3].shape, generator=torch.Generator().manual_seed(1))
    pools[3].mul_(f.cuda())                                            # every value 2^-30 to 2^-10 of what it was
    ref[1] *= f[..., None]
    q = _q(5, 4, D, dtype, 21)
    pools[3].mul_(2.0 ** 20), ref[1].mul_(2.0 ** 20)
    o = _call(sv, q, pools, table, seq_len, [3, 0])
    want = su.attention_ref(q, *ref, table, seq_len, _i32([3, 0]))
    big = want[0].abs().amax(-1, keepdim=True)
    off = (o["out"].cpu().double() - want[0]).abs() - RTOL[dtype] * want[0].abs() - 2.0 ** -12 * big
    assert off.max() < (2.0 ** -24 if dtype == torch.float16 else 0), off.max()


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_a_row_does_not_see(sv, quant, dtype, D):
    """Scales that are not finite, or codes that are no numbers, at the last
    new token: rows in front of it are what they are without."""
    L, nd, P = [150, 77], [4, 2], 16
    keep = torch.tensor([0, 1, 2, 3, 5, 6])
    for what in ("scale", "inf") + (("code",) if quant == cu.E4M3 else ()):
        pools, ref, table, seq_len = cu.make_coded_pages(L, P, 2, D, dtype, quant, 10)
        q = _q(8, 6, D, dtype, 10)
        want = su.attention_ref(q, *ref, table, seq_len, _i32(nd))
        for b, n in enumerate(L):
            p = table[b, (n - 1) // P].long()
            if what == "code":
                pools[2].view(torch.uint8)[p, :, (n - 1) % P, 5] = 0xFF
            else:
                for s in (pools[1], pools[3]):
                    s[p, :, (n - 1) % P] = torch.nan if what == "scale" else torch.inf
        o = _call(sv, q, pools, table, seq_len, nd)
        _near(o, want, dtype, keep)
        got = o["out"][[4, 7]]
        assert torch.isnan(got[..., 5]).all() if what == "code" else not torch.isfinite(got).any() or what == "inf"


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("heads", [2, 8])
def test_many_rows_next_to_few(sv, heads, quant, dtype):
    """Two and three row tiles, of which some sequences leave the higher ones
    empty; then a value without a number (or its scale) at the last new token,
    which only the last rows see."""
    L, nd, P = [290, 70, 9, 300], [7, 0, 1, 8], 16
    pools, ref, table, seq_len = cu.make_coded_pages(L, P, 2, 128, dtype, quant, 12)
    N = sum(n + 1 for n in nd)
    q = _q(N, heads, 128, dtype, 12)
    want = su.attention_ref(q, *ref, table, seq_len, _i32(nd))
    _near(_call(sv, q, pools, table, seq_len, nd), want, dtype)
    _near(_call(sv, q, pools, table, seq_len, nd, window=40), su.attention_ref(q, *ref, table, seq_len, _i32(nd), window=40), dtype)
    last = [7, 8, 10, 19]
    for b, n in enumerate(L):
        p = table[b, (n - 1) // P].long()
        if quant == cu.E4M3:
            pools[2].view(torch.uint8)[p, :, (n - 1) % P, 77] = 0x7F
        else:
            pools[3][p, :, (n - 1) % P] = torch.nan
    o = _call(sv, q, pools, table, seq_len, nd)
    _near(o, want, dtype, [i for i in range(N) if i not in last])
    assert torch.isnan(o["out"][last][..., 77]).all()


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("falling", [False, True])
def test_scores_that_grow_or_fall(sv, falling, D, quant, dtype):
    """As the test of that name for shared prefixes, which has the errors."""
    for nd, L in (([8, 0, 7], [1500, 40, 900]), ([0], [1500])):
        made = cu.make_coded_pages(L, 32, 1, D, dtype, quant, 32)
        cu.ramp_keys(*made, 32, quant, falling)
        q = _q(sum(n + 1 for n in nd), 4, D, dtype, 32)
        q[:, :, 0] = 200.0
        _near(_call(sv, q, made[0], made[2], made[3], nd), su.attention_ref(q, *made[1], made[2], made[3], _i32(nd)), dtype)


@pytest.mark.parametrize("quant", [cu.E4M3, cu.INT8])
def test_rows_that_see_nothing(sv, quant):
    o = _run(sv, [0, 3, 40, 0], [0, 5, 2, 3], 8, 2, 128, 16, torch.bfloat16, quant, seed=9)
    assert (o["out"][0] == 0).all() and (o["lse"][0] == -torch.inf).all()


def test_strided_codes(sv):
    """A layer of a cache of layers; scales between others."""
    pools, ref, table, seq_len = cu.make_coded_pages([100, 40], 16, 2, 64, torch.bfloat16, cu.INT8, 13)
    n = pools[0].shape[0]
    wide = torch.full((3, n, 4, 16, 64), 127, dtype=torch.int8, device="cuda")
    wide[1, :, ::2] = pools[0]
    scales = torch.full((n, 3, 2, 16), torch.nan, device="cuda")
    scales[:, 1] = pools[1]
    q = _q(5, 8, 64, torch.bfloat16, 13)
    o = _call(sv, q, [wide[1, :, ::2], scales[:, 1], pools[2], pools[3]], table, seq_len, [3, 0])
    _near(o, su.attention_ref(q, *ref, table, seq_len, _i32([3, 0])), torch.bfloat16)


def test_far_offsets(sv):
    """Codes beyond 2^32 bytes from the pool's start."""
    P, KV, D = 64, 8, 128
    n = (1 << 32) // (P * KV * D) + 40
    pools, ref, table, seq_len = cu.make_coded_pages([300], P, KV, D, torch.bfloat16, cu.INT8, 15, extra=0)
    far = torch.arange(n - pools[0].shape[0], n, dtype=torch.int32).cuda()
    k = torch.empty(n, KV, P, D, dtype=torch.int8, device="cuda")
    s = torch.empty(n, KV, P, device="cuda")
    k[far.long()], s[far.long()] = pools[2], pools[3]
    at = table.clone()
    at[0] = far[table[0].long()]
    q = _q(3, 16, D, torch.bfloat16, 15)
    o = _call(sv, q, [k, s, k, s], at, seq_len, [2])
    _near(o, su.attention_ref(q, ref[1], ref[1], table, seq_len, _i32([2])), torch.bfloat16)


@pytest.mark.parametrize("quant,dtype", KINDS)
def test_a_round_over_the_cache(sv, quant, dtype):
    """Reserve, norms and rotation into the cache, attention, commit; then
    another round.  The reference reads the cache back."""
    H, KV, D, P = 8, 2, 128, 16
    c = sv.PagedCache(layers=2, num_pages=40, page_size=P, kv_heads=KV, head_dim=D, max_seqs=4, max_pages=12, dtype=dtype, device="cuda", quant=quant)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.view(torch.uint8).fill_(0xFF)
    g = torch.Generator().manual_seed(3)
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    w = torch.ones(D, dtype=dtype, device="cuda")
    seqs = _i32([2, 0, 3])
    for nd, accepted in (([90, 30, 0], [90, 30, 0]), ([4, 0, 5], [2, 0, -1]), ([3, 200, 1], [1, 0, 1])):
        n = sum(x + 1 for x in nd)
        r = c.reserve(seqs, _i32([x + 1 for x in nd]), n, want_positions=True)
        refused = nd[1] == 200
        assert r["status"].tolist() == [0, 512 if refused else 0, 0]
        qkv = (torch.randn(n, H + 2 * KV, D, generator=g) * 2).to(dtype).cuda()
        q = c.write_rotated(1, qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:], r["slots"], r["positions"], f, q_weight=w, k_weight=w)
        o = c.attend(1, q, _i32(nd), seqs, start=r["start"], want_lse=True)
        assert o["status"].tolist() == r["status"].tolist()
        rows, kept = [], [b for b in range(3) if not (refused and b == 1)]
        at = 0
        for b in range(3):
            rows += list(range(at, at + nd[b] + 1)) if b in kept else []
            at += nd[b] + 1
        codes = [c.k[1].view(torch.uint8).cpu(), c.v[1].view(torch.uint8).cpu()]
        grid = torch.from_numpy(cu.e4m3_values()) if quant == cu.E4M3 else torch.arange(256).to(torch.uint8).view(torch.int8).double()
        held = [grid[x.long()] * s[1].cpu().double()[..., None] for x, s in zip(codes, (c.k_scale, c.v_scale))]
        want = su.attention_ref(q[torch.tensor(rows).cuda()], *held, c.page_table, c.seq_len, _i32([nd[b] for b in kept]), seqs=seqs[kept].cpu())
        _near({"out": o["out"][torch.tensor(rows).cuda()], "lse": o["lse"][torch.tensor(rows).cuda()]}, want, dtype)
        if refused:
            assert torch.isnan(o["out"][5 - 1:5 - 1 + 201]).all()
        c.commit(seqs, _i32(nd), _i32(accepted), start=r["start"])
    assert c.seq_len.tolist() == [31 + 1, 0, 91 + 3 + 2, 1 + 0 + 2]


def test_streams_graph_and_repeats(sv):
    dtype = torch.bfloat16
    pools, _, table, seq_len = cu.make_coded_pages([3000, 40, 700], 16, 2, 128, dtype, cu.E4M3, 17)
    q, nd = _q(9, 8, 128, dtype, 17), [3, 0, 3]
    want = _call(sv, q, pools, table, seq_len, nd)
    torch.cuda.synchronize()
    got = [_call(sv, q, pools, table, seq_len, nd, stream=s) for s in [torch.cuda.Stream() for _ in range(2)] for _ in range(2)]
    torch.cuda.synchronize()
    for o in got:
        for key in want:
            assert torch.equal(want[key], o[key])
    ndt = _i32(nd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = sv.paged_attention(q, pools[0], pools[2], table, seq_len, ndt, k_scale=pools[1], v_scale=pools[3], want_lse=True)
    for i in range(4):
        q.copy_(_q(9, 8, 128, dtype, 30 + i))
        seq_len.copy_(_i32([3000 - 500 * i, 40 - i, 700 - 100 * i]))
        fresh = _call(sv, q, pools, table, seq_len, nd)
        graph.replay()
        torch.cuda.synchronize()
        for key in fresh:
            assert torch.equal(fresh[key], o[key]), (i, key)


def test_refusals(sv):
    dtype = torch.bfloat16
    pools, _, table, seq_len = cu.make_coded_pages([100, 40], 16, 2, 64, dtype, cu.E4M3, 20)
    q = _q(3, 4, 64, dtype, 20)

    def call(k=pools[0], ks=pools[1], v=pools[2], vs=pools[3]):
        return sv.paged_attention(q, k, v, table, seq_len, _i32([1, 0]), k_scale=ks, v_scale=vs)
    call()
    for kw in (dict(k=pools[0].view(torch.int8)), dict(k=pools[0].view(torch.uint8), v=pools[2].view(torch.uint8)),
               dict(k=torch.zeros(pools[0].shape, dtype=dtype, device="cuda"))):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(TypeError):
        call(ks=None, vs=None)
    for kw in (dict(ks=None), dict(vs=pools[3].double()), dict(ks=pools[1][:1]), dict(ks=pools[1].cpu()),
               dict(ks=pools[1].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)
    odd = torch.empty(pools[1].numel() + 1, device="cuda")[1:].view(pools[1].shape)
    with pytest.raises(sv.VerifyError):
        call(ks=odd)
    c = sv.PagedCache(1, 4, 16, 2, 64, 2, 2, dtype=dtype, device="cuda", quant="int8")
    with pytest.raises(TypeError):
        c.attend(0, q.half(), _i32([1, 0]))
