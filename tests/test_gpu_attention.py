"""Attention over a paged cache on the GPU against a float64 form.

Tolerances.  The result is rounded once to the 16-bit type (u = 2^-9 relative
for bfloat16, 2^-12 for float16, half a unit).  Before that: a score is a
float32 sum of D exact products, off by at most D 2^-24 sum |q_d k_d| scale;
with |q|, |k| entries of size 1 to 2 that is below A = 256 2^-24 * 2 * 16 *
1.45 < 2^-11 in the exponent for head_dim 256 in the worst case and near its
square root in practice; it moves every weight by that factor at most, hence
the result by 2 A max |v|.  The two 16-bit halves of a weight hold it to 2^-17
(bfloat16) or 2^-22, and the float32 sums over L positions in runs of 32 add
(L / 32 + 40) 2^-24.  With max |v| < 6 over these sizes the absolute part
stays below ATOL = 6 * (2^-10 + 2^-17 + 2^-16) < 2^-7 as a worst case; the
tests ask for a quarter of the worst case, 2^-9, plus the rounding
(RTOL = 2^-8 and 2^-11, one unit)."""
import numpy as np
import pytest
import torch

from . import serving_util as su

pytestmark = pytest.mark.gpu

RTOL = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
ATOL = 2.0 ** -9


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


def _near(o, ref, dtype):
    out, lse = ref
    got = o["out"].cpu().double()
    assert not torch.isnan(got).any()
    d = (got - out).abs() - RTOL[dtype] * out.abs()
    assert d.max() < ATOL, d.max()
    if o["lse"] is not None:
        l = o["lse"].cpu().double()
        assert torch.equal(torch.isinf(l), torch.isinf(lse))
        fine = ~torch.isinf(lse)
        assert (l - lse).abs()[fine].max() < 2.0 ** -10 if fine.any() else True


def _run(sv, L, nd, H, KV, D, P, dtype, seed=0, layout="head", std=1.0, **kw):
    k, v, table, seq_len = su.make_pages(L, P, KV, D, dtype, seed, layout)
    q = _q(sum(n + 1 for n in nd), H, D, dtype, seed, std)
    o = sv.paged_attention(q, k, v, table, seq_len, _i32(nd), want_lse=True, **kw)
    torch.cuda.synchronize()
    assert not o["status"].cpu().any()
    _near(o, su.attention_ref(q, k, v, table, seq_len, _i32(nd), kw.get("seqs"), kw.get("scale"), kw.get("window", 0)), dtype)
    return o


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 1000])
def test_one_token(sv, L, D, dtype):
    _run(sv, [L], [0], 8, 2, D, 16, dtype, seed=L)


@pytest.mark.parametrize("P", [16, 32, 64, 1024])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_pages_and_layouts(sv, P, layout):
    _run(sv, [700, 5, 130, 1], [3, 0, 5, 0], 4, 2, 128, P, torch.bfloat16, seed=P, layout=layout)


@pytest.mark.parametrize("H,KV", [(1, 1), (7, 1), (16, 16), (32, 8), (15, 3), (40, 2), (64, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_groups(sv, H, KV, D):
    _run(sv, [300, 65, 129], [4, 0, 1], H, KV, D, 32, torch.bfloat16, seed=H)


@pytest.mark.parametrize("nd", [[8, 8, 8], [0, 31, 2], [63, 0, 0], [16, 15, 17], [128, 1, 0]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_ragged_rows(sv, nd, dtype):
    """Row tiles that are full, cut, and more than one to a sequence."""
    _run(sv, [300, 290, 200], nd, 8, 2, 128, 16, dtype, seed=sum(nd))


@pytest.mark.parametrize("window", [1, 2, 16, 31, 100, 128, 129, 1000, 2147483647])
def test_window(sv, window):
    _run(sv, [1, 40, 300, 777], [0, 5, 8, 3], 8, 4, 64, 16, torch.bfloat16, seed=window % 1000, window=window)


def test_scale_and_sharp_softmax(sv):
    _run(sv, [500, 200], [2, 1], 4, 1, 128, 16, torch.bfloat16, seed=1, scale=0.5)
    _run(sv, [500, 200], [2, 1], 4, 1, 128, 16, torch.bfloat16, seed=2, scale=0.0)
    _run(sv, [500, 200], [2, 1], 4, 1, 64, 16, torch.float16, seed=3, std=4.0)


def test_many_parts(sv):
    """Long sequences that many blocks share, next to short ones."""
    _run(sv, [20011, 3, 1, 9000], [2, 0, 0, 8], 8, 2, 128, 16, torch.bfloat16, seed=5)
    _run(sv, [30000], [0], 2, 1, 64, 64, torch.float16, seed=6)
    _run(sv, [12345], [3], 4, 1, 256, 32, torch.bfloat16, seed=7)


def test_many_sequences(sv):
    r = np.random.RandomState(0)
    L = r.randint(1, 60, 1300).tolist()
    _run(sv, L, [int(r.randint(0, min(4, x))) for x in L], 2, 2, 64, 16, torch.bfloat16, seed=8)


def test_rows_that_see_nothing(sv):
    """Sequences of length zero, and with fewer tokens than rows."""
    o = _run(sv, [0, 3, 40, 0], [0, 5, 2, 3], 8, 2, 128, 16, torch.bfloat16, seed=9)
    assert (o["out"][0] == 0).all() and (o["lse"][0] == -torch.inf).all()
    assert (o["out"][1:4] == 0).all() and torch.isfinite(o["lse"][4:]).sum() == 6 * 8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", ["nan", "inf", "lowest"])
def test_what_a_row_does_not_see(sv, dtype, D, what):
    """The last new token's key and value are not finite (or the type's
    lowest): the rows in front of it are what they are without it."""
    L, nd, P = [150, 77], [4, 2], 16
    k, v, table, seq_len = su.make_pages(L, P, 2, D, dtype, 10)
    q = _q(8, 6, D, dtype, 10)
    x = {"nan": torch.nan, "inf": torch.inf, "lowest": torch.finfo(dtype).min}[what]
    ref = su.attention_ref(q, k, v, table, seq_len, _i32(nd))
    for b, n in enumerate(L):
        p = table[b, (n - 1) // P].long()
        k[p, :, (n - 1) % P], v[p, :, (n - 1) % P] = x, x
    o = sv.paged_attention(q, k, v, table, seq_len, _i32(nd), want_lse=True)
    keep = torch.tensor([0, 1, 2, 3, 5, 6])
    got = {"out": o["out"][keep.cuda()], "lse": o["lse"][keep.cuda()]}
    _near(got, (ref[0][keep], ref[1][keep]), dtype)
    if what == "nan":
        assert torch.isnan(o["out"][[4, 7]]).all()
    # behind a window: the old end of the cache is not finite
    k, v, table, seq_len = su.make_pages(L, P, 2, D, dtype, 11)
    ref = su.attention_ref(q, k, v, table, seq_len, _i32(nd), window=20)
    for b, n in enumerate(L):
        for j in range(n - nd[b] - 20):
            p = table[b, j // P].long()
            k[p, :, j % P], v[p, :, j % P] = x, x
    _near(sv.paged_attention(q, k, v, table, seq_len, _i32(nd), want_lse=True, window=20), ref, dtype)


@pytest.mark.parametrize("P", [16, 64])
def test_pages_behind_a_window_may_be_gone(sv, P):
    dtype, L, nd, window = torch.bfloat16, [700, 300, 90], [3, 0, 5], 100
    k, v, table, seq_len = su.make_pages(L, P, 2, 64, dtype, 18)
    q = _q(11, 4, 64, dtype, 18)
    want = sv.paged_attention(q, k, v, table, seq_len, _i32(nd), window=window, want_lse=True)
    for b, n in enumerate(L):
        gone = max(0, n - nd[b] - window) // P                   # pages no row sees anything of
        table[b, :gone] = torch.tensor([-1, 1 << 30], dtype=torch.int32).repeat(99)[:gone].cuda()
    got = sv.paged_attention(q, k, v, table, seq_len, _i32(nd), window=window, want_lse=True)
    assert not got["status"].any()
    for key in want:
        assert torch.equal(want[key], got[key])
    _near(got, su.attention_ref(q, k, v, table.clamp(min=0).clamp(max=k.shape[0] - 1), seq_len, _i32(nd), window=window), dtype)
    table[0, max(0, 700 - 3 - window) // P] = -1                   # the first page that is seen
    assert sv.paged_attention(q, k, v, table, seq_len, _i32(nd), window=window)["status"].tolist() == [1024, 0, 0]


@pytest.mark.parametrize("D,H", [(64, 64), (128, 40), (128, 64), (256, 20)])
def test_largest_batch(sv, D, H):
    """4096 sequences of a few tokens, every height of row tile."""
    dtype = torch.float16
    L = [1 + i % 3 for i in range(4096)]
    k, v, table, seq_len = su.make_pages(L, 16, 1, D, dtype, 19)
    q, nd = _q(4096, H, D, dtype, 19), torch.zeros(4096, dtype=torch.int32, device="cuda")
    o = sv.paged_attention(q, k, v, table, seq_len, nd, want_lse=True)
    assert not o["status"].any()
    kk = torch.stack([k[table[:, 0].long(), 0, j] for j in range(3)], 1).cpu().double()
    vv = torch.stack([v[table[:, 0].long(), 0, j] for j in range(3)], 1).cpu().double()
    hide = torch.arange(3)[None] >= torch.tensor(L)[:, None]
    s = torch.matmul(q.cpu().double(), kk.transpose(1, 2).contiguous()) * D ** -0.5
    s = s.masked_fill(hide[:, None], -torch.inf)
    ref = torch.matmul(torch.softmax(s, -1), vv.masked_fill(hide[:, :, None], 0.0))
    _near(o, (ref, torch.logsumexp(s, -1)), dtype)


def test_slots(sv):
    """Sequences in another order than their slots, one slot twice."""
    dtype = torch.bfloat16
    k, v, table, seq_len = su.make_pages([100, 40, 0, 333], 16, 2, 128, dtype, 12)
    q, nd, seqs = _q(9, 4, 128, dtype, 12), _i32([2, 0, 0, 3]), _i32([3, 0, 3, 1])
    o = sv.paged_attention(q, k, v, table, seq_len, nd, seqs=seqs, want_lse=True)
    _near(o, su.attention_ref(q, k, v, table, seq_len, nd, seqs=seqs.cpu()), dtype)


def test_strided_inputs(sv):
    """q as a slice of a fused projection, a layer of a cache of layers, a
    table wider than what is used."""
    dtype = torch.bfloat16
    k, v, table, seq_len = su.make_pages([100, 40], 16, 2, 64, dtype, 13)
    wide = torch.full((2, table.shape[1] + 5), 12345, dtype=torch.int32).cuda()
    wide[:, :table.shape[1]] = table
    layers = torch.full((3, *k.shape), torch.nan, dtype=dtype).cuda()
    layers[1] = k
    qkv = torch.full((5, 8 + 2 + 2, 64), torch.nan, dtype=dtype).cuda()
    qkv[:, :8] = _q(5, 8, 64, dtype, 13)
    nd = _i32([3, 0])
    o = sv.paged_attention(qkv[:, :8], layers[1], v, wide[:, :table.shape[1]], seq_len, nd, want_lse=True)
    _near(o, su.attention_ref(qkv[:, :8], k, v, table, seq_len, nd), dtype)


def test_status(sv):
    dtype = torch.bfloat16
    k, v, table, seq_len = su.make_pages([100, 40, 64, 30], 16, 2, 128, dtype, 14)
    q = _q(7, 4, 128, dtype, 14)
    nd = _i32([2, 0, 1, 0])
    good = sv.paged_attention(q, k, v, table, seq_len, nd, want_lse=True)
    # a bad page behind the last token is not looked at
    t2 = table.clone()
    t2[1, 3:] = 1 << 30
    same = sv.paged_attention(q, k, v, t2, seq_len, nd, want_lse=True)
    for key in good:
        assert torch.equal(good[key], same[key])
    t2[0, 4], t2[2, 3] = k.shape[0], -5
    l2 = seq_len.clone()
    l2[3] = table.shape[1] * 16 + 1
    o = {a: b.cpu() for a, b in sv.paged_attention(q, k, v, t2, l2, nd, want_lse=True).items()}
    assert o["status"].tolist() == [1024, 0, 1024, 512]
    assert torch.equal(o["out"][3], good["out"][3].cpu()) and torch.isfinite(o["out"][3]).all()
    for rows in (slice(0, 3), slice(4, 7)):
        assert torch.isnan(o["out"][rows]).all() and torch.isnan(o["lse"][rows]).all()
    o = sv.paged_attention(q, k, v, table, seq_len, nd, seqs=_i32([0, 4, -1, 3]), want_lse=True)
    assert o["status"].tolist() == [0, 256, 256, 0] and torch.isnan(o["out"][3:6]).all()
    assert torch.equal(o["out"][:3], good["out"][:3]) and torch.equal(o["out"][6], good["out"][6])
    l2 = seq_len.clone()
    l2[0] = -1
    assert sv.paged_attention(q, k, v, table, l2, nd)["status"].tolist() == [512, 0, 0, 0]
    for bad in ([2, 0, 1, 1], [2, 0, 2, -1], [2147483647, 0, 1, 0], [1, 0, 1, 0]):
        o = sv.paged_attention(q, k, v, table, seq_len, _i32(bad), want_lse=True)
        assert o["status"].tolist() == [1] * 4 and torch.isnan(o["out"]).all() and torch.isnan(o["lse"]).all()


def test_far_offsets(sv):
    """Pages whose elements lie beyond 2^32 bytes (and 2^31 elements) from the pool's start."""
    dtype, P, KV, D = torch.bfloat16, 64, 8, 128
    pages = (1 << 32) // (P * KV * D) + 40                        # 2^32 elements, 8 GiB
    k = torch.empty(pages, KV, P, D, dtype=dtype, device="cuda")
    ks, vs, table, seq_len = su.make_pages([300], P, KV, D, dtype, 15, extra=0)
    far = torch.arange(pages - ks.shape[0], pages, dtype=torch.int32).cuda()
    k[far.long()] = ks
    at = table.clone()
    at[0] = far[table[0].long()]
    q = _q(3, 16, D, dtype, 15)
    o = sv.paged_attention(q, k, k, at, seq_len, _i32([2]), want_lse=True)
    _near(o, su.attention_ref(q, ks, ks, table, seq_len, _i32([2])), dtype)


def test_empty_batch(sv):
    k, v, table, seq_len = su.make_pages([10], 16, 1, 64, torch.bfloat16, 16)
    o = sv.paged_attention(_q(0, 4, 64, torch.bfloat16, 1), k, v, table, seq_len, _i32([]))
    assert o["out"].shape == (0, 4, 64)


def test_streams_graph_and_repeats(sv):
    dtype = torch.bfloat16
    k, v, table, seq_len = su.make_pages([3000, 40, 700], 16, 2, 128, dtype, 17)
    q, nd = _q(9, 8, 128, dtype, 17), _i32([3, 0, 3])
    want = sv.paged_attention(q, k, v, table, seq_len, nd, want_lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [sv.paged_attention(q, k, v, table, seq_len, nd, want_lse=True, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for o in got:
        for key in want:
            assert torch.equal(want[key], o[key])
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = sv.paged_attention(q, k, v, table, seq_len, nd, want_lse=True)
        graphs.append((graph, o))
    for i in range(4):
        q.copy_(_q(9, 8, 128, dtype, 30 + i))
        seq_len.copy_(_i32([3000 - 500 * i, 40 - i, 700 - 100 * i]))
        fresh = sv.paged_attention(q, k, v, table, seq_len, nd, want_lse=True)
        for graph, o in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, o in graphs:
            for key in fresh:
                assert torch.equal(fresh[key].nan_to_num(), o[key].nan_to_num()), (i, key)


def test_refused_by_the_host(sv):
    dtype = torch.bfloat16
    k, v, table, seq_len = su.make_pages([100, 40], 16, 2, 64, dtype, 20)
    q, nd = _q(3, 4, 64, dtype, 20), _i32([1, 0])

    def call(**kw):
        a = dict(q=q, k_pages=k, v_pages=v, page_table=table, seq_len=seq_len, num_draft=nd)
        extra = {n: kw.pop(n) for n in ("seqs", "window", "scale") if n in kw}
        a.update(kw)
        return sv.paged_attention(*a.values(), **extra)
    call()
    for kw in (dict(q=q[0]), dict(q=q[:, :, :32]), dict(v_pages=v[:, :1]), dict(page_table=table.long()), dict(page_table=table.t()),
               dict(seq_len=seq_len[:1]), dict(q=q.cpu()), dict(k_pages=k.cpu()), dict(seqs=_i32([0])), dict(num_draft=_i32([0, 0, 0])),
               dict(window=1 << 32), dict(k_pages=k.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=q.float()), dict(k_pages=k.half()), dict(num_draft=nd.long()), dict(seqs=nd.float())):
        with pytest.raises(TypeError):
            call(**kw)
    odd = torch.empty(q.numel() + 1, dtype=dtype, device="cuda")[1:].view(q.shape)
    for kw in (dict(window=-1), dict(scale=float("nan")), dict(q=odd), dict(q=torch.cat([q, q[:, :1]], 1)), dict(q=q[:1]),
               dict(page_table=table[:, :0])):
        with pytest.raises(sv.VerifyError):
            call(**kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_far_below_the_largest(sv, dtype):
    """One key far above 30000 others whose weights, 2.7e-5 of its own and
    below the smallest normal float16, still make up almost half of the sum."""
    L, D = 30001, 64
    k, v, table, seq_len = su.make_pages([L], 16, 1, D, dtype, 21)
    pages = table[0].long()
    k.zero_(), v.fill_(1.0)
    k[pages[0], 0, 0, 0] = 10.5 * 8
    v[pages[0], 0, 0] = -1.0
    q = torch.zeros(1, 2, D, dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    o = sv.paged_attention(q, k, v, table, seq_len, _i32([0]), want_lse=True)
    small = (L - 1) * np.exp(-10.5)
    want = (small - 1) / (small + 1)
    assert (o["out"].double().cpu() - want).abs().max() < abs(want) * RTOL[dtype] + 2.0 ** -12
    assert abs(o["lse"][0, 0].item() - (10.5 + np.log1p(small))) < 1e-4


def test_rows_without_a_sequence(sv):
    k, v, table, seq_len = su.make_pages([10], 16, 1, 64, torch.bfloat16, 16)
    with pytest.raises(sv.VerifyError):
        sv.paged_attention(_q(3, 4, 64, torch.bfloat16, 1), k, v, table, seq_len, _i32([]))
