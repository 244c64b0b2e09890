"""Token log probabilities on the GPU against a float64 form of their own.

Tolerances.  With c = log2(e)/T, a term's exponent y = x c - round(M c) is
formed with one rounding, so 2^y is off by |y| 2^-24 ln 2 relative plus the
exponential's one unit; M c itself is rounded, |M c| 2^-24 absolute in log2
units, shared by every term and by the token's own y.  c is off by at most
2^-23 relative (the constant's and the division's rounding), which moves y by
|y| 2^-23.  Sums of V positive terms over a tree of depth <= 64 + 20 are off by
84 * 2^-24 relative.  With |y| <= Y (the spread of the row in log2 units) the
log probability is therefore off by less than ln 2 (Y 2^-22 + |M c| 2^-23) +
2^-17, and the entropy (a mean of such y) by the same.  TOL(Y) below is that
bound, doubled for the spread of the terms that carry the sums."""
import numpy as np
import pytest
import torch

from . import serving_util as su

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rejection_sampling_verify_06_amd as m
    return m


def _tol(logits, vocab, temperature):
    x = logits.detach().cpu().double()[:, :vocab]
    big = torch.where(x.abs() < 1e30, x, 0.0).abs().max().item()
    t = 1.0 if temperature is None else float(temperature.min())
    return 2 * (3 * big / t * 1.4427 * 2.0 ** -22 + 2.0 ** -17)


def _check(sv, logits, tokens, temperature=None, vocab=None, top=0, **kw):
    V = logits.shape[1] if vocab is None else vocab
    o = sv.token_logprobs(logits, tokens, top=top, temperature=temperature, vocab=vocab, **kw)
    torch.cuda.synchronize()
    ref = su.logprobs_ref(logits, None if tokens is None else tokens.cpu().numpy(),
                          None if temperature is None else temperature.cpu().numpy(), V, top)
    tol = _tol(logits, V, temperature)
    assert not o["status"].cpu().numpy().any()
    for k in ("logprob", "entropy"):
        if o[k] is not None:
            got = o[k].cpu().double().numpy()
            np.testing.assert_allclose(got, ref[k], rtol=2e-6, atol=tol, err_msg=k)
    if tokens is not None:
        assert np.array_equal(o["rank"].cpu().numpy(), ref["rank"])
    assert np.array_equal(o["top_tokens"].cpu().numpy(), ref["top_tokens"])
    got = o["top_logprobs"].cpu().double().numpy()
    same = np.isinf(ref["top_logprobs"])
    assert np.array_equal(np.isinf(got), same)
    np.testing.assert_allclose(got[~same], ref["top_logprobs"][~same], rtol=2e-6, atol=tol)
    return o


def _rows(R, V, dtype, seed, scale=3.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, V + pad, generator=g) * scale
    return x.to(dtype).cuda(), torch.randint(0, V, (R,), generator=g).to(torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 255, 256, 257, 1000, 16383, 16384, 16385, 16391, 40003])
def test_vocab_edges(sv, V, dtype):
    logits, tok = _rows(5, V, dtype, V)
    _check(sv, logits, tok, top=min(V, 20))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,off", [(0, 1), (1, 0), (3, 2), (5, 7), (8, 0)])
def test_strides_and_alignment(sv, pad, off, dtype):
    """Rows that start at every offset from a 16-byte boundary, the columns
    behind the vocabulary holding the largest values."""
    R, V = 9, 5003
    g = torch.Generator().manual_seed(pad * 10 + off)
    flat = torch.full((R * (V + pad) + off,), 1e4)
    view = flat[off:].view(R, V + pad)
    view[:, :V] = torch.randn(R, V, generator=g) * 2
    logits = flat.to(dtype).cuda()[off:].view(R, V + pad)
    tok = torch.randint(0, V, (R,), generator=g).to(torch.int32).cuda()
    _check(sv, logits, tok, vocab=V, top=17)


@pytest.mark.parametrize("top", [0, 1, 2, 31, 63, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_top_counts(sv, top, dtype):
    logits, tok = _rows(4, 70001, dtype, top)
    _check(sv, logits, tok, top=top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties(sv, dtype):
    """Constant rows, rows of few values, rows whose best tokens fill one
    segment, ascending and descending rows, and 0 against -0."""
    V = 33000
    i = torch.arange(V, dtype=torch.float32)
    rows = torch.stack([
        torch.zeros(V), (i % 3), (i % 1000 == 999).float(), torch.where((i >= 500) & (i < 700), 5.0, 0.0),
        i / V, -i / V, torch.where(i % 2 == 0, 0.0, -0.0), torch.where(i == V - 1, 1.0, -0.0),
        torch.where(i < V - 40, -1.0, 2.0), torch.full((V,), -7.0)]).to(dtype).cuda()
    tok = torch.tensor([0, 5, V - 1, 600, 17, 3, 1, 0, V - 1, 12], dtype=torch.int32).cuda()
    _check(sv, rows, tok, top=64)


@pytest.mark.parametrize("top", [5, 64])
def test_ties_over_a_long_row(sv, top):
    """Rows of one and of few values, longer than what is listed at a time."""
    V = 600001
    i = torch.arange(V, dtype=torch.float32)
    rows = torch.stack([torch.zeros(V), i % 2, (i > V - 30).float(), (i % 9973 == 5).float() * 2,
                        torch.where(i < 300000, -torch.inf, -3.0)]).to(torch.bfloat16).cuda()
    tok = torch.tensor([7, 8, V - 1, 5, V - 1], dtype=torch.int32).cuda()
    _check(sv, rows, tok, top=top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_and_extreme_values(sv, dtype):
    """-inf and the type's lowest value as masks, all but one token masked,
    every token at the lowest value, huge spreads."""
    V, lo = 3001, torch.finfo(dtype).min
    g = torch.Generator().manual_seed(3)
    x = torch.randn(7, V, generator=g).to(dtype)
    x[0, 5:] = -torch.inf
    x[1, 5:] = lo
    x[2, :] = -torch.inf
    x[2, 77] = 1.5
    x[3, :] = lo
    x[4, ::2] = -torch.inf
    x[5, 100] = 80.0
    x[6, :] = lo
    x[6, 1] = 3.0
    tok = torch.tensor([2, 3, 77, 9, 1, 100, 1], dtype=torch.int32)
    _check(sv, x.cuda(), tok.cuda(), top=8)
    # the masked tokens' own log probabilities
    o = sv.token_logprobs(x.cuda(), torch.tensor([9, 9, 9, 0, 0, 0, 0], dtype=torch.int32).cuda())
    lp = o["logprob"].cpu()
    assert lp[0] == -torch.inf and lp[2] == -torch.inf and lp[4] == -torch.inf and lp[1] < -1e30 and lp[6] < -1e30
    assert abs(lp[3].item() + np.log(V)) < 1e-5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale,T", [(3.0, 1e-6), (3.0, 1e-4), (1e4, 1e-6), (1e5, 0.05), (1e30, 1.0), (1e38, 1.0), (3.0, 1e30)])
def test_extreme_exponents(sv, dtype, scale, T):
    """Logits over temperature far beyond what an exponential holds: one token
    takes all, or all are alike; whole numbers in units of the scale, so that
    gaps are either 0 or large."""
    g = torch.Generator().manual_seed(int(scale) % 1000 + 7)
    x = (torch.randint(-3, 3, (6, 40000), generator=g).float() * scale).to(dtype)
    x[:, 100], x[1, 30000], x[2, 0] = 3 * scale, 3 * scale, 3 * scale
    tok = torch.tensor([100, 30000, 5, 100, 6, 100], dtype=torch.int32)
    t = torch.full((6,), T)
    o = sv.token_logprobs(x.cuda(), tok.cuda(), temperature=t.cuda(), top=3)
    ref = su.logprobs_ref(x, tok.numpy(), t.numpy(), 40000, 3)
    assert not o["status"].any() and np.array_equal(o["top_tokens"].cpu().numpy(), ref["top_tokens"])
    for k in ("logprob", "entropy", "top_logprobs"):
        got, want = o[k].cpu().double().numpy(), ref[k]
        want = np.where(want < -3.4e38, -np.inf, want)          # beyond float32
        assert np.array_equal(np.isinf(got), np.isinf(want)), (k, got, want)
        fine = np.isfinite(want)
        np.testing.assert_allclose(got[fine], want[fine], rtol=2e-6, atol=1e-5)


@pytest.mark.parametrize("base", [0.0, 7.0e5, 7.2682e5, 7.28e5, 1e6, -7.2682e5])
def test_references_near_their_border(sv, base):
    """Rows whose scaled maximum lies on both sides of the size up to which it
    is rounded, in one row: the parts meet on the same scale."""
    g = torch.Generator().manual_seed(4)
    x = (torch.randint(0, 64, (2, 60000), generator=g) * 0.0625 + base).float()
    x[:, :20000] -= 2.0
    tok = torch.tensor([17, 40000], dtype=torch.int32)
    o = sv.token_logprobs(x.cuda(), tok.cuda(), top=4)
    ref = su.logprobs_ref(x, tok.numpy(), None, 60000, 4)
    # y = x c - round(M c) is rounded once, below 2^-19 here: log2 S and y together are off by 2^-18
    for k in ("logprob", "entropy", "top_logprobs"):
        np.testing.assert_allclose(o[k].cpu().double().numpy(), ref[k], rtol=2e-6, atol=2.0 ** -17)


def test_skipped_rows_are_not_read(sv):
    logits, tok = _rows(40, 4096, torch.bfloat16, 8)
    tok[::3] = -1
    poisoned = logits.clone()
    poisoned[::3] = torch.nan
    o = _check(sv, logits, tok, top=5)
    p = sv.token_logprobs(poisoned, tok, top=5)
    for k in o:
        assert torch.equal(o[k], p[k]), k
    assert (p["logprob"][::3] == 0).all() and (p["top_tokens"][::3] == -1).all()


def test_temperature_and_status(sv):
    logits, tok = _rows(8, 20011, torch.float32, 9)
    t = torch.tensor([0.3, 1.0, 2.0, 0.05, 7.0, 1.2, 0.7, 1.0])
    _check(sv, logits, tok, temperature=t.cuda(), top=6)
    t[1], t[2], t[3], t[4] = 0.0, -1.0, torch.nan, torch.inf
    tok[5] = 20011
    logits[6, 123] = torch.nan
    logits[7, 4] = torch.inf
    o = {k: v.cpu() for k, v in sv.token_logprobs(logits, tok, temperature=t.cuda(), top=6).items()}
    assert o["status"].tolist() == [0, 8, 8, 8, 8, 32, 64, 64]
    assert torch.isnan(o["logprob"][1:]).all() and torch.isnan(o["entropy"][1:]).all()
    assert (o["top_tokens"][1:] == -1).all() and torch.isnan(o["top_logprobs"][1:]).all() and (o["rank"][1:] == 0).all()
    assert torch.isfinite(o["logprob"][0]) and (o["top_tokens"][0] >= 0).all()
    allinf = torch.full((1, 100), -torch.inf).cuda()
    assert sv.token_logprobs(allinf, top=3)["status"].item() == 64


def test_without_tokens_and_optional_outputs(sv):
    logits, tok = _rows(6, 9001, torch.bfloat16, 10)
    a = _check(sv, logits, tok, top=4)
    b = sv.token_logprobs(logits, None, top=4)
    assert b["logprob"] is None and b["rank"] is None
    assert torch.equal(a["entropy"], b["entropy"]) and torch.equal(a["top_tokens"], b["top_tokens"])
    c = sv.token_logprobs(logits, tok, want_entropy=False, want_rank=False, want_status=False)
    assert c["entropy"] is None and c["rank"] is None and c["status"] is None and c["top_tokens"].shape == (6, 0)
    assert torch.equal(c["logprob"], a["logprob"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_vocabulary(sv, dtype):
    logits, tok = _rows(2, 2097152, dtype, 11)
    _check(sv, logits, tok, top=64)


def test_many_rows(sv):
    """More blocks than one grid dimension holds."""
    logits, tok = _rows(70000, 33, torch.bfloat16, 12)
    _check(sv, logits, tok, top=3)


def test_no_rows(sv):
    o = sv.token_logprobs(torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), top=2)
    assert o["logprob"].shape == (0,) and o["top_tokens"].shape == (0, 2)


def test_streams_and_repeats(sv):
    """The same bits from two calls at once on two streams."""
    logits, tok = _rows(64, 50021, torch.bfloat16, 13)
    want = sv.token_logprobs(logits, tok, top=20)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [sv.token_logprobs(logits, tok, top=20, stream=s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for g in got:
        for k in want:
            assert torch.equal(want[k], g[k]), k


def test_graph(sv):
    logits, tok = _rows(16, 30011, torch.bfloat16, 14)
    sv.token_logprobs(logits, tok, top=5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = sv.token_logprobs(logits, tok, top=5)
    for i in range(4):
        new, t = _rows(16, 30011, torch.bfloat16, 20 + i)
        logits.copy_(new)
        tok.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = sv.token_logprobs(new, t, top=5)
        for k in o:
            assert torch.equal(want[k], o[k]), (i, k)


def test_after_a_verify_call(sv):
    """A round's emitted tokens scored on its own target rows: the log
    probability of an accepted token is the log of the verify call's p."""
    from workloads import make_random_batch
    from . import gpu_util as gu
    b = make_random_batch(21, B=24, V=3000, kmax=6, dtype="bf16", modes=(0,))
    d = gu.batch_to_device(b, torch, 0)
    out = sv.verify(d["target"], d["draft"], d["draft_tokens"], d["num_draft"], d["temperature"], d["mode"], seed=5,
                    want_pq=True, seq_ids=d["seq_ids"])
    n = d["num_draft"].long() + 1
    T = torch.repeat_interleave(d["temperature"], n)
    lp = sv.token_logprobs(d["target"][:, :b.vocab], out["emitted"], temperature=T, top=3)
    torch.cuda.synchronize()
    emitted, A = out["emitted"].cpu().numpy(), out["accepted_len"].cpu().numpy()
    p, got = out["p_at"].cpu().double().numpy(), lp["logprob"].cpu().double().numpy()
    ranks = lp["rank"].cpu().numpy()
    od = ot = scored = 0
    for s, K in enumerate(b.num_draft):
        for i in range(K + 1):
            assert (ranks[ot + i] > 0) == (emitted[ot + i] >= 0)
            if i < A[s]:
                assert abs(np.exp(got[ot + i]) - p[od + i]) < 1e-5
                scored += 1
        od, ot = od + K, ot + K + 1
    assert scored > 0
