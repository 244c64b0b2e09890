"""Attention of batches whose sequences share prefixes on the GPU, against
float64 over each whole sequence.

Tolerances as for the call without groups: the prefix's part of a row is kept
in float32 (its value, and log2 of its sum of weights) and joined as any other
part, which adds a few 2^-24."""
import numpy as np
import pytest
import torch

from . import coded_util as cu
from . import serving_util as su

pytestmark = pytest.mark.gpu

RTOL = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
ATOL = 2.0 ** -9
KINDS = [(q, d) for q in (None, cu.E4M3, cu.INT8) for d in (torch.bfloat16, torch.float16)]


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


def _call(sv, q, made, nd, **kw):
    pools, _, table, seq_len, groups, prefix = made
    a = dict(k_scale=pools[1], v_scale=pools[3], groups=groups, prefix_len=prefix, want_lse=True)
    a.update(kw)
    return sv.paged_attention(q, pools[0], pools[2], a.pop("table", table), a.pop("seq_len", seq_len), _i32(nd), **a)


def _run(sv, groups, nd, H, KV, D, P, dtype, quant=None, seed=0, std=1.0, **kw):
    made = cu.make_shared(groups, P, KV, D, dtype, quant, seed)
    q = _q(sum(n + 1 for n in nd), H, D, dtype, seed, std)
    o = _call(sv, q, made, nd, **kw)
    torch.cuda.synchronize()
    assert not o["status"].cpu().any()
    _near(o, su.attention_ref(q, *made[1], made[2], made[3], _i32(nd), None, kw.get("scale")), dtype)
    return o, made, q


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [1, 16, 31, 127, 128, 129, 1000])
def test_branches(sv, prefix, D, quant, dtype):
    """Three branches of a sequence, a few tokens of their own."""
    _run(sv, [(prefix, [1, 40, 9])], [0, 3, 1], 8, 2, D, 16, dtype, quant, seed=prefix)


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("H,KV,D", [(1, 1, 64), (16, 16, 64), (32, 8, 128), (15, 3, 256), (40, 2, 64), (64, 1, 128)])
def test_head_groups(sv, H, KV, D, quant, dtype):
    _run(sv, [(300, [5, 65, 20]), (77, [4])], [4, 0, 1, 3], H, KV, D, 32, dtype, quant, seed=H)


@pytest.mark.parametrize("quant", [None, cu.E4M3, cu.INT8])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows(sv, quant, D):
    """Groups of dozens of sequences: hundreds of rows a key head, tiles that
    are full and cut, next to small groups."""
    r = np.random.RandomState(D)
    groups = [(700, r.randint(9, 60, 40).tolist()), (33, [9, 12]), (260, r.randint(9, 60, 21).tolist())]
    nd = [int(x) for x in r.randint(0, 9, 63)]
    _run(sv, groups, nd, 8, 2, D, 16, torch.bfloat16, quant, seed=1)
    _run(sv, groups, nd, 6, 6, D, 64, torch.float16, quant, seed=2)


@pytest.mark.parametrize("P", [16, 64, 1024])
def test_prefixes_of_every_kind(sv, P):
    """None, whole pages, parts of a page, longer than the own part; groups of
    one and empty groups."""
    groups = [(0, [50, 3]), (64, [1]), (1024, [1, 700]), (5, [5]), (2048 + 13, [20, 9, 9, 9])]
    made = cu.make_shared(groups, P, 2, 64, torch.bfloat16, None, 3)
    nd = [2, 0, 0, 0, 5, 4, 0, 8, 1, 0]
    q = _q(sum(n + 1 for n in nd), 4, 64, torch.bfloat16, 3)
    ref = su.attention_ref(q, *made[1], made[2], made[3], _i32(nd))
    _near(_call(sv, q, made, nd), ref, torch.bfloat16)
    first, prefix = made[4].tolist(), made[5].tolist()
    first.insert(3, first[2])                                                # an empty group, whose prefix may be anything
    first = [0] + first + [first[-1]]
    prefix.insert(2, -7)
    prefix = [99999] + prefix + [1 << 30]
    o = _call(sv, q, made, nd, groups=_i32(first), prefix_len=_i32(prefix))
    assert not o["status"].any()
    _near(o, ref, torch.bfloat16)
    # less than they share is no mistake
    _near(_call(sv, q, made, nd, prefix_len=_i32([0, 3, 1000, 0, 129])), ref, torch.bfloat16)


@pytest.mark.parametrize("quant", [None, cu.INT8])
def test_long_prefix(sv, quant):
    _run(sv, [(20011, [3, 1, 9, 200])], [2, 0, 8, 1], 8, 2, 128, 16, torch.bfloat16, quant, seed=5)
    _run(sv, [(9000, [9] * 30)], [8] * 30, 8, 2, 64, 16, torch.float16, quant, seed=6)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_few_rows_behind_long_prefixes(sv, dtype):
    """20 to 24 rows of a key head in the tiles made for many."""
    _run(sv, [(9000, [5, 9, 3]), (8001, [7, 2])], [1, 2, 0, 3, 0], 64, 16, 128, 16, dtype, seed=8)


def test_sharp_softmax_and_scales(sv):
    """Rows whose weight lies all in the prefix, or all in their own part."""
    _run(sv, [(500, [20, 3])], [2, 1], 4, 1, 64, 16, torch.float16, seed=3, std=4.0)
    _run(sv, [(500, [20, 3])], [2, 1], 4, 1, 128, 16, torch.bfloat16, seed=2, scale=0.0)
    for dtype in (torch.bfloat16, torch.float16):
        made = cu.make_shared([(100, [30, 30])], 16, 1, 64, dtype, None, 4)
        k, table = made[0][0], made[2]
        for pos in (40, 110):
            x = k.clone()
            for b in range(2):
                x[table[b, pos // 16].long(), 0, pos % 16, 0] = 400.0
            q = _q(2, 2, 64, dtype, 4)
            q[:, :, 0] = 8.0
            o = _call(sv, q, ([x, None, made[0][2], None], *made[1:]), [0, 0])
            for b in range(2):
                want = made[0][2][table[b, pos // 16].long(), 0, pos % 16]
                assert torch.equal(o["out"][b], want[None].expand(2, -1))


@pytest.mark.parametrize("quant,dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("falling", [False, True])
def test_scores_that_grow_or_fall(sv, falling, D, quant, dtype):
    """Along 1500 keys the scores grow (or fall) by some 3 * 200 / sqrt(D) = 37 to
    75, a few units with every tile, so that the rows' maximum moves many times,
    now by less and now by more than what the weights may grow by; many rows
    (tiles of 128) and few.  A score's float32 sum is off by some 8 * 600 * 2^-24
    before the scale of at most 1 / 8, a weight by 2^-14 of itself."""
    for own, group in (([30, 9, 50] * 7, 4), ([30, 9], 1)):
        made = cu.make_shared([(1500, own)], 32, 1, D, dtype, quant, 31)
        cu.ramp_keys(made[0], made[1], made[2], made[3], 32, quant, falling)
        nd = [i % 4 for i in range(len(own))]
        q = _q(sum(n + 1 for n in nd), group, D, dtype, 31)
        q[:, :, 0] = 200.0
        o = _call(sv, q, made, nd)
        assert not o["status"].any()
        _near(o, su.attention_ref(q, *made[1], made[2], made[3], _i32(nd)), dtype)


@pytest.mark.parametrize("quant,dtype", KINDS)
def test_what_is_not_finite(sv, quant, dtype):
    """A key of the prefix, then one of a sequence's own, that is not finite:
    the rows that see it are not, the others stay what they are."""
    groups, nd = [(100, [10, 20]), (50, [5, 7])], [2, 0, 1, 0]
    made = cu.make_shared(groups, 16, 2, 128, dtype, quant, 7)
    q = _q(7, 4, 128, dtype, 7)
    ref = su.attention_ref(q, *made[1], made[2], made[3], _i32(nd))
    for b, pos, rows in ((0, 37, [0, 1, 2, 3]), (0, 109, [2]), (3, 55, [6])):
        pools = [None if x is None else x.clone() for x in made[0]]
        page = made[2][b, pos // 16].long()
        for i in (0, 2):
            if quant is None:
                pools[i][page, :, pos % 16] = torch.nan
            else:
                pools[i + 1][page, :, pos % 16] = torch.nan
        o = _call(sv, q, (pools, *made[1:]), nd)
        assert torch.isnan(o["out"][rows]).all() and not o["status"].any()
        _near(o, ref, dtype, [i for i in range(7) if i not in rows])


def test_refused_sequences(sv):
    dtype = torch.bfloat16
    groups, nd = [(100, [10, 20, 8]), (0, [40]), (50, [5, 7])], [2, 0, 1, 0, 1, 0]
    made = cu.make_shared(groups, 16, 2, 64, dtype, None, 8)
    pools, _, table, seq_len, first, prefix = made
    q = _q(10, 4, 64, dtype, 8)
    ref = su.attention_ref(q, *made[1], table, seq_len, _i32(nd))
    good = _call(sv, q, made, nd)
    begin = [0, 3, 4, 6, 7, 9, 10]

    def check(status, **kw):
        n = kw.pop("nd", nd)
        o = _call(sv, q, made, n, **kw)
        assert o["status"].tolist() == status
        for b, s in enumerate(status):
            rows = slice(begin[b], begin[b + 1])
            if s:
                assert torch.isnan(o["out"][rows]).all() and torch.isnan(o["lse"][rows]).all()
            else:
                assert torch.equal(o["out"][rows], good["out"][rows]) and torch.equal(o["lse"][rows], good["lse"][rows])

    _near(good, ref, dtype)
    check([0] * 6)
    for bad in (-1, 1 << 30, 2147483647):
        check([512, 512, 512, 0, 0, 0], prefix_len=_i32([bad, 0, 50]))
    check([0, 0, 0, 512, 0, 0], prefix_len=_i32([100, 40, 50]))              # the new token is in it
    t = table.clone()
    t[1, 2] = t[1, 6]                                                         # another page than the leader's
    check([0, 1024, 0, 0, 0, 0], table=t)
    t = table.clone()
    t[:3, 2] = pools[0].shape[0]                                              # shared, and outside the pool
    check([1024] * 3 + [0] * 3, table=t)
    t = table.clone()
    t[2, 6] = -1                                                              # its own page (the copy of the prefix's last)
    check([0, 0, 1024, 0, 0, 0], table=t)
    t = table.clone()
    t[0, 6] = -1                                                              # the leader's: the prefix's end
    check([1024] * 3 + [0] * 3, table=t)
    l = seq_len.clone()
    l[1] = 100
    check([0, 512, 0, 0, 0, 0], seq_len=l)                                    # its new token is in the prefix
    l = seq_len.clone()
    l[0] = 99                                                                 # the leader does not have the prefix
    check([512] * 3 + [0] * 3, seq_len=l)
    l[0], l[4] = -1, table.shape[1] * 16 + 1
    check([512] * 3 + [0, 512, 512], seq_len=l)
    for seqs, status in (([0, 6, 2, 3, 4, 5], [0, 256, 0, 0, 0, 0]), ([-1, 1, 2, 3, 4, 5], [256, 256, 256, 0, 0, 0])):
        check(status, seqs=_i32(seqs))
    # sequences that sit the round out, the first of a group among them
    start = (seq_len - _i32(nd) - 1)
    start[0], start[5] = -1, -1
    check([512, 0, 0, 0, 0, 512], start=start)
    # layouts that do not add up
    for kw in (dict(nd=[2, 0, 1, 0, 1, 1]), dict(nd=[2, 0, 2, -1, 1, 0]), dict(groups=_i32([0, 3, 4, 5])), dict(groups=_i32([1, 3, 4, 6])),
               dict(groups=_i32([0, 4, 3, 6])), dict(groups=_i32([0, 3, 7, 6])), dict(groups=_i32([0, -1, 4, 6]))):
        o = _call(sv, q, made, kw.pop("nd", nd), **kw)
        assert o["status"].tolist() == [1] * 6 and torch.isnan(o["out"]).all() and torch.isnan(o["lse"]).all()


def test_slots_strides_and_one_sequence_twice(sv):
    dtype = torch.bfloat16
    made = cu.make_shared([(200, [10, 20, 30]), (90, [5, 6])], 16, 2, 128, dtype, None, 9)
    pools, _, table, seq_len, _, _ = made
    seqs, nd = [3, 4, 3, 1, 0, 2], [0, 2, 1, 3, 0, 1]
    N = sum(nd) + 6
    qkv = torch.full((N, 12, 128), torch.nan, dtype=dtype, device="cuda")
    qkv[:, :8] = _q(N, 8, 128, dtype, 9)
    wide = torch.full((5, table.shape[1] + 3), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    layers = torch.full((3, *pools[0].shape), torch.nan, dtype=dtype, device="cuda")
    layers[1] = pools[0]
    o = sv.paged_attention(qkv[:, :8], layers[1], pools[2], wide[:, :table.shape[1]], seq_len, _i32(nd), seqs=_i32(seqs), groups=_i32([0, 3, 6]),
                           prefix_len=_i32([90, 200]), want_lse=True)
    assert not o["status"].any()
    _near(o, su.attention_ref(qkv[:, :8], *made[1], table, seq_len, _i32(nd), seqs=seqs), dtype)


def test_largest_batch(sv):
    """4096 sequences in 4096 groups, in one, and in 300."""
    dtype, H, D = torch.bfloat16, 4, 64
    made = cu.make_shared([(40, [1 + i % 5 for i in range(4096)])], 16, 2, D, dtype, None, 10)
    pools, _, table, seq_len, _, _ = made
    q, nd = _q(4096, H, D, dtype, 10), [0] * 4096
    want = sv.paged_attention(q, pools[0], pools[2], table, seq_len, _i32(nd), want_lse=True)
    for first, prefix in ((list(range(4097)), [40] * 4096), ([0, 4096], [40]), ([0] + list(range(10, 3000, 10)) + [4096], [40, 33] * 150)):
        o = _call(sv, q, made, nd, groups=_i32(first), prefix_len=_i32(prefix[:len(first) - 1]))
        assert not o["status"].any()
        assert ((o["out"].double() - want["out"].double()).abs() <= 2.0 ** -7 * want["out"].double().abs() + 1e-4).all()
        assert (o["lse"] - want["lse"]).abs().max() < 1e-5


@pytest.mark.parametrize("quant", [None, cu.E4M3])
def test_rounds_of_forks(sv, quant):
    """A prompt, forked; rounds of the branches over the cache, as they would
    be used: reserve, norms and rotation into the cache, attention over the shared
    prefix, commit.  One branch sits a round out."""
    dtype, H, KV, D, P = torch.bfloat16, 8, 2, 128, 16
    c = sv.PagedCache(layers=1, num_pages=64, page_size=P, kv_heads=KV, head_dim=D, max_seqs=6, max_pages=24, dtype=dtype, device="cuda", quant=quant)
    g = torch.Generator().manual_seed(11)
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    w = torch.ones(D, dtype=dtype, device="cuda")

    def into(r, n):
        qkv = (torch.randn(n, H + 2 * KV, D, generator=g) * 2).to(dtype).cuda()
        return c.write_rotated(0, qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:], r["slots"], r["positions"], f, q_weight=w, k_weight=w)

    for s, n in ((0, 203), (3, 64)):
        into(c.reserve(_i32([s]), _i32([n]), n, want_positions=True), n)
    assert c.fork(_i32([0, 0, 3]), _i32([1, 2, 4])).tolist() == [0, 0, 0]
    seqs, groups, prefix = _i32([2, 0, 1, 3, 4]), _i32([0, 3, 5]), _i32([203, 64])
    for nd, accepted in (([3, 0, 5, 1, 1], [1, 0, 5, 0, 1]), ([2, 2, 300, 0, 0], [2, 0, 0, 0, -1]), ([4, 4, 4, 4, 4], [4, 3, 2, 1, 0])):
        n = sum(nd) + 5
        r = c.reserve(seqs, _i32([x + 1 for x in nd]), n, want_positions=True)
        q = into(r, n)
        o = c.attend(0, q, _i32(nd), seqs, start=r["start"], groups=groups, prefix_len=prefix, want_lse=True)
        plain = c.attend(0, q, _i32(nd), seqs, start=r["start"], want_lse=True)
        assert torch.equal(o["status"], r["status"]) and torch.equal(o["status"], plain["status"])
        assert o["status"].tolist() == [0, 0, 512 if nd[2] == 300 else 0, 0, 0]
        assert torch.equal(o["out"].isnan(), plain["out"].isnan())
        a, b = o["out"].nan_to_num().double(), plain["out"].nan_to_num().double()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -11).all()
        assert (o["lse"].nan_to_num() - plain["lse"].nan_to_num()).abs().max() < 1e-4
        assert not c.commit(seqs, _i32(nd), _i32(accepted), start=r["start"])[[0, 1, 3, 4]].any()


def test_streams_graphs_and_repeats(sv):
    dtype = torch.bfloat16
    made = cu.make_shared([(1000, [60] * 12), (300, [50, 9])], 16, 2, 128, dtype, None, 12)
    pools, _, table, seq_len, first, prefix = made
    nd = [4] * 14
    q = _q(70, 8, 128, dtype, 12)
    want = _call(sv, q, made, nd)
    torch.cuda.synchronize()
    got = [_call(sv, q, made, nd, stream=s) for s in [torch.cuda.Stream() for _ in range(2)] for _ in range(2)]
    torch.cuda.synchronize()
    for o in got:
        for key in want:
            assert torch.equal(want[key], o[key])
    ndt, graphs = _i32(nd), []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = sv.paged_attention(q, pools[0], pools[2], table, seq_len, ndt, groups=first, prefix_len=prefix, want_lse=True)
        graphs.append((graph, o))
    for i in range(4):
        q.copy_(_q(70, 8, 128, dtype, 30 + i))
        seq_len.copy_(_i32([1060 - 3 * i] * 12 + [350, 309 - 2 * i]))
        prefix.copy_(_i32([1000 - 300 * i, 300]))
        fresh = _call(sv, q, made, nd)
        assert fresh["status"].tolist() == [0] * 13 + [512 if 309 - 2 * i < 305 else 0]
        for graph, o in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, o in graphs:
            for key in fresh:
                assert torch.equal(fresh[key].nan_to_num(), o[key].nan_to_num()), (i, key)


def test_refused_by_the_host(sv):
    made = cu.make_shared([(40, [10, 20])], 16, 2, 64, torch.bfloat16, None, 13)
    q = _q(2, 4, 64, torch.bfloat16, 13)
    _call(sv, q, made, [0, 0])
    for kw in (dict(groups=None), dict(prefix_len=None), dict(groups=_i32([0, 1, 2])), dict(groups=made[4].cpu()), dict(prefix_len=made[5].cpu())):
        with pytest.raises(ValueError):
            _call(sv, q, made, [0, 0], **kw)
    for kw in (dict(groups=made[4].long()), dict(prefix_len=made[5].float())):
        with pytest.raises(TypeError):
            _call(sv, q, made, [0, 0], **kw)
    for kw in (dict(window=8), dict(groups=_i32([0, 1, 2, 2]), prefix_len=_i32([0, 0, 0]))):
        with pytest.raises(sv.VerifyError):
            _call(sv, q, made, [0, 0], **kw)
