"""The serving operators around the verify step, as cases that can be timed: log probabilities of given tokens, attention of
a round's new tokens over a paged key-value cache, and the cache's own operations (reserve, write, commit, fork, release,
compact).

``run`` computes a case either in its plain form (elementary torch operations, in 32 bits) or, with ``own`` set, through the
package's entry points.  Sizes that vary from sequence to sequence follow from the case alone; the values follow from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one sequence's round over a small vocabulary, logprobs of what was emitted with 5 alternatives: latency
        dict(name="logprobs_one", op="logprobs", batch=1, k=5, vocab=32000, dtype="bf16", top=5, emitted=True, temp=False),
        # the logprobs a service returns for a whole round of a large batch, 20 alternatives each
        dict(name="logprobs_round", op="logprobs", batch=256, k=8, vocab=152064, dtype="bf16", top=20, emitted=True, temp=False),
        # every row of a batch scored, float32 logits, a temperature, an odd vocabulary, no alternatives
        dict(name="logprobs_score_f32", op="logprobs", batch=32, k=5, vocab=128255, dtype="f32", top=0, emitted=False, temp=True),
        # one new token of one short sequence: latency
        dict(name="attn_one_token", op="attn", batch=1, k=0, max_len=777, heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", window=0),
        # a round of 5 drafts over a batch of mixed lengths
        dict(name="attn_round", op="attn", batch=32, k=5, max_len=8192, heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", window=0),
        # two long documents, 8 drafts each
        dict(name="attn_long", op="attn", batch=2, k=8, max_len=131072, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16", window=0),
        # many short sequences, every head its own keys, small heads
        dict(name="attn_short_mha", op="attn", batch=256, k=3, max_len=1000, heads=16, kv_heads=16, dim=64, page=32, dtype="f16", window=0),
        # one key head for all query heads, wide heads, a sliding window
        dict(name="attn_mqa_window", op="attn", batch=16, k=4, max_len=20000, heads=8, kv_heads=1, dim=256, page=16, dtype="bf16", window=4096),
        # the cache's side of one decode round: the last round's tokens dropped, K + 1 reserved and written, the rejected ones dropped
        dict(name="cache_round", op="round", batch=32, k=5, max_len=2048, layers=4, kv_heads=8, dim=128, page=16, dtype="bf16"),
        # prompts of up to 1024 tokens enter the cache
        dict(name="cache_prompts", op="round", batch=16, k=1023, max_len=64, layers=4, kv_heads=8, dim=128, page=16, dtype="bf16"),
        # every sequence branches into 3, each branch takes 2 tokens of its own (copy on write), the branches are released
        dict(name="cache_branch", op="branch", batch=64, ways=3, k=1, max_len=500, layers=8, kv_heads=8, dim=128, page=16, dtype="bf16"),
        # half of the sequences leave, the rest moves to the front of the pool, new ones enter
        dict(name="cache_compact", op="compact", batch=64, max_len=512, layers=4, kv_heads=8, dim=128, page=16, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "attn", "attn", "attn", "round", "branch", "compact"])
    if op == "logprobs":
        vocab = _log_int(rng, 1000, 152064)
        most = max(1, min(1400, int(1400 * 152064 * 0.45 / vocab)))
        k = rng.randint(0, 8)
        return dict(op=op, batch=_log_int(rng, 1, max(1, most // (k + 1))), k=k, vocab=vocab, dtype=rng.choice(["bf16", "f32"]),
                    top=rng.choice([0, 1, 5, 20, 31]), emitted=rng.random() < 0.5, temp=rng.random() < 0.5)
    if op == "attn":
        dim = rng.choice([64, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8])
        k = rng.randint(0, 8)
        max_len = _log_int(rng, 16, 65536)
        tokens = (1 << 27) // (kv * dim)
        return dict(op=op, batch=max(1, min(256, _log_int(rng, 1, max(1, tokens // max_len)))), k=k, max_len=max_len,
                    heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f16"]),
                    window=rng.choice([0, 0, 0, 100, 1024]))
    page = rng.choice([16, 32, 64])
    kv, dim, layers = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.randint(1, 4)
    if op == "round":
        k = rng.choice([0, 1, 3, 5, 8, rng.randint(9, 700)])
        return dict(op=op, batch=_log_int(rng, 1, 128 if k < 9 else 16), k=k, max_len=_log_int(rng, 1, 1000), layers=layers, kv_heads=kv,
                    dim=dim, page=page, dtype=rng.choice(["bf16", "f16"]))
    if op == "branch":
        return dict(op=op, batch=_log_int(rng, 1, 64), ways=rng.randint(1, 3), k=rng.randint(0, 5), max_len=_log_int(rng, 1, 500), layers=layers,
                    kv_heads=kv, dim=dim, page=page, dtype=rng.choice(["bf16", "f16"]))
    return dict(op=op, batch=_log_int(rng, 2, 64), max_len=_log_int(rng, 16, 500), layers=layers, kv_heads=kv, dim=dim, page=page,
                dtype=rng.choice(["bf16", "f16"]))


def _sizes(case):
    """The per-sequence sizes of a case, from the case alone."""
    key = [case["batch"], case.get("k", 0), case.get("max_len", 1), case.get("vocab", 1), case.get("heads", 1), case.get("page", 1)]
    r = np.random.RandomState(key)
    B = case["batch"]
    s = {}
    kmax = case.get("k", 0)
    s["num_draft"] = np.full(B, kmax) if B == 1 else r.randint(min(1, kmax), kmax + 1, B)
    s["accepted"] = np.floor(r.rand(B) * (s["num_draft"] + 1)).astype(np.int64)
    if "max_len" in case:
        m = case["max_len"]
        lens = np.full(B, m) if B == 1 else r.randint(max(1, m // 8), m + 1, B)
        if case["op"] == "attn":
            lens = np.maximum(lens, s["num_draft"] + 1)
        s["len"] = lens
    return s


def work(case):
    z = _sizes(case)
    n = z["num_draft"] + 1
    if case["op"] == "logprobs":
        rows = int((z["accepted"] + 1).sum()) if case["emitted"] else int(n.sum())
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * case["vocab"] * e + int(n.sum()) * (4 + 16 + 8 * case["top"]), "flops": rows * case["vocab"] * 8}
    kv, D = case["kv_heads"], case["dim"]
    if case["op"] == "attn":
        L = z["len"]
        first = np.maximum(0, L - n + 1 - case["window"]) if case["window"] else 0 * L
        rows = int(n.sum())
        i = np.arange(case["k"] + 1)[None, :]
        seen = np.where(i < n[:, None], (L - n)[:, None] + i + 1, 0)
        if case["window"]:
            seen = np.minimum(seen, case["window"])
        return {"bytes": int((L - first).sum()) * kv * D * 4 + rows * case["heads"] * (4 * D + 4), "flops": int(seen.sum()) * case["heads"] * D * 4}
    token = case["layers"] * kv * D * 4
    page, P = token * case["page"], case["page"]
    if case["op"] == "round":
        return {"bytes": int(n.sum()) * token * 2, "flops": 0}
    if case["op"] == "branch":
        copied = int((z["len"] % P != 0).sum()) * case["ways"]
        pages = int((-(-z["len"] // P)).sum()) * case["ways"]
        return {"bytes": copied * page * 2 + pages * 12, "flops": 0}
    half = -(-z["len"] // P)
    moved = min(int(half[0::2].sum()), int(half[1::2].sum()))
    return {"bytes": moved * page * 2 + int(half.sum()) * 12, "flops": 0}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _dev(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(device=DEV, dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = _sizes(case)
    s = dict(case=case)
    make = {"logprobs": _prepare_logprobs, "attn": _prepare_attn}.get(case["op"], _prepare_cache)
    make(case, z, s, g)
    return s


def _prepare_logprobs(case, z, s, g):
    n = z["num_draft"] + 1
    N, V = int(n.sum()), case["vocab"]
    ld = V if case["dtype"] == "bf16" else V + 1
    x = torch.randn(N, ld, generator=g, device=DEV)
    rank = torch.randperm(ld, generator=g, device=DEV) + 1
    x -= 1.1 * rank.log()                                   # Zipf-shaped, as a language model's logits are
    s["logits"] = x.to(DTYPES[case["dtype"]])
    # the tokens: drawn from the rows' own distributions
    u = torch.rand(N, ld, generator=g, device=DEV)
    x -= torch.log(-torch.log(u.clamp_(1e-12, 1 - 1e-7)))
    tok = x[:, :V].argmax(1).to(torch.int32)
    if case["emitted"]:                                     # a round's packed rows: x_0 .. x_{A-1}, y, then -1
        at = np.arange(N) - np.repeat(np.cumsum(n) - n, n)
        tok[_dev(at > np.repeat(z["accepted"], n), torch.bool)] = -1
    s["tokens"] = tok
    s["temperature"] = 0.5 + torch.rand(N, generator=g, device=DEV) if case["temp"] else None


def _prepare_attn(case, z, s, g):
    B, P, D, H = case["batch"], case["page"], case["dim"], case["kv_heads"]
    n, L = z["num_draft"] + 1, z["len"]
    dt = DTYPES[case["dtype"]]
    pages = -(-L // P)
    total = int(pages.sum())
    N = int(n.sum())
    s["k"] = torch.empty(total + 3, H, P, D, dtype=dt, device=DEV).normal_(generator=g)
    s["v"] = torch.empty(total + 3, H, P, D, dtype=dt, device=DEV).normal_(generator=g)
    s["q"] = torch.empty(N, case["heads"], D, dtype=dt, device=DEV).normal_(std=2.0, generator=g)
    ids = torch.randperm(total + 3, generator=g, device=DEV)[:total].to(torch.int32)
    table = torch.full((B, int(pages.max())), -1, dtype=torch.int32, device=DEV)
    table[_dev(np.arange(table.shape[1])[None, :] < pages[:, None], torch.bool)] = ids
    s["table"], s["len"], s["num_draft"] = table, _dev(L), _dev(z["num_draft"])


def _prepare_cache(case, z, s, g):
    """A pool whose pages lie in random order, and what the pass hands to it."""
    B, P, D, H, Y = case["batch"], case["page"], case["dim"], case["kv_heads"], case["layers"]
    dt, op = DTYPES[case["dtype"]], case["op"]
    n, L = z["num_draft"] + 1, z["len"].copy()
    keep = z["accepted"] + 1
    slots = B * (1 + case["ways"]) if op == "branch" else B
    held = L + (keep if op == "round" else 0)               # a round finds the last one's committed tokens in the cache
    pages = -(-held // P)
    if op == "compact":                                     # the first group's pages in front of the second's
        first = np.arange(B) % 2 == 0
        order = np.argsort(~first, kind="stable")
        ids = np.empty(int(pages.sum()), np.int64)
        starts = np.cumsum(pages) - pages
        at = 0
        for b in order:
            ids[starts[b]:starts[b] + pages[b]] = np.arange(at, at + pages[b])
            at += pages[b]
        num_pages = at + 8
    else:
        extra = int((-(-(L + n) // P) - pages).clip(0).sum())
        if op == "branch":
            extra = int(((-(-(L + n) // P) - L // P) * (case["ways"] + 1)).sum())
        num_pages = int(pages.sum()) + extra + 8
        ids = torch.randperm(num_pages, generator=g, device=DEV).cpu().numpy()[:int(pages.sum())]
    width = int((-(-(L + n + (keep if op == "round" else 0)) // P)).max()) + 1
    table = np.full((slots, width), -1, np.int64)
    table[:B][np.arange(width)[None, :] < pages[:, None]] = ids
    ref = np.zeros(num_pages, np.int64)
    ref[ids] = 1
    lens = np.zeros(slots, np.int64)
    lens[:B] = held
    k = torch.empty(Y, num_pages, H, P, D, dtype=dt, device=DEV).normal_(generator=g)
    v = torch.empty(Y, num_pages, H, P, D, dtype=dt, device=DEV).normal_(generator=g)
    s["seqs"] = _dev(np.random.RandomState(B).permutation(B) if op == "round" else np.arange(B))
    pick = s["seqs"].cpu().numpy()
    if op == "round":
        s["kept"], s["num_new"], s["num_draft"] = _dev(keep[pick]), _dev(n[pick]), _dev((n - 1)[pick])
        s["accepted"], s["total"] = _dev((keep - 1)[pick]), int(n.sum())
        s["k_new"] = torch.empty(Y, s["total"], H, D, dtype=dt, device=DEV).normal_(generator=g)
        s["v_new"] = torch.empty(Y, s["total"], H, D, dtype=dt, device=DEV).normal_(generator=g)
    elif op == "branch":
        s["parents"] = _dev(np.repeat(np.arange(B), case["ways"]))
        s["children"] = _dev(B + np.arange(B * case["ways"]))
        s["num_new"], s["total"] = _dev(np.repeat(n, case["ways"])), int(n.sum()) * case["ways"]
    else:
        for t in (0, 1):
            s["group%d" % t] = _dev(np.arange(t, B, 2))
            s["back%d" % t], s["total%d" % t] = _dev(L[t::2]), int(L[t::2].sum())
        s["turn"] = 0
    if own:
        import rejection_sampling_verify_06_amd as sv
        c = sv.PagedCache(layers=Y, num_pages=num_pages, page_size=P, kv_heads=H, head_dim=D, max_seqs=slots, max_pages=width,
                          dtype=dt, device=DEV)
        c.k.copy_(k), c.v.copy_(v), c.page_table.copy_(_dev(table)), c.seq_len.copy_(_dev(lens)), c.refcount.copy_(_dev(ref))
        s["cache"] = c
    else:
        s.update(k=k, v=v, table=_dev(table), len=_dev(lens), ref=_dev(ref))


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(s):
    return {"logprobs": _run_logprobs, "attn": _run_attn, "round": _run_round, "branch": _run_branch, "compact": _run_compact}[s["case"]["op"]](s)


def _run_logprobs(s):
    c = s["case"]
    if own:
        import rejection_sampling_verify_06_amd as sv
        o = sv.token_logprobs(s["logits"], s["tokens"], top=c["top"], temperature=s["temperature"], vocab=c["vocab"])
        return [o["logprob"], o["entropy"], o["rank"], o["top_tokens"], o["top_logprobs"]]
    V, top, tok = c["vocab"], c["top"], s["tokens"]
    raw = s["logits"][:, :V].float() + 0.0
    x = raw if s["temperature"] is None else raw / s["temperature"][:, None]
    x = x - x.amax(1, keepdim=True)
    e = x.exp()
    total = e.sum(1)
    skip = tok < 0
    at = tok.clamp(min=0).long()[:, None]
    log_total = total.log()
    logprob = torch.where(skip, 0.0, x.gather(1, at)[:, 0] - log_total)
    entropy = torch.where(skip, 0.0, log_total - (e * x).sum(1) / total)
    rank = torch.where(skip, 0, (raw > raw.gather(1, at)).sum(1) + 1).to(torch.int32)
    bits = raw.view(torch.int32)
    bits = bits ^ ((bits >> 31) & 0x7FFFFFFF)                # ordered like the values; the lower index first on ties
    keys = (bits.long() << 32) | (0xFFFFFFFF - torch.arange(V, device=DEV))
    ids = 0xFFFFFFFF - (keys.topk(top, dim=1).values & 0xFFFFFFFF)
    top_lp = torch.where(skip[:, None], -math.inf, x.gather(1, ids) - log_total[:, None])
    ids = torch.where(skip[:, None], -1, ids).to(torch.int32)
    return [logprob, entropy, rank, ids, top_lp]


def _run_attn(s):
    c = s["case"]
    if own:
        import rejection_sampling_verify_06_amd as sv
        o = sv.paged_attention(s["q"], s["k"], s["v"], s["table"], s["len"], s["num_draft"], window=c["window"], want_lse=True)
        return [o["out"], o["lse"]]
    q, table = s["q"], s["table"].clamp(min=0).long()
    B, H, D, R = c["batch"], c["kv_heads"], c["dim"], c["k"] + 1
    G, N = c["heads"] // H, q.shape[0]
    n = s["num_draft"].long() + 1
    off = n.cumsum(0) - n
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n, output_size=N)
    i = torch.arange(N, device=DEV) - off[seq]
    rows = (off[:, None] + torch.arange(R, device=DEV)).clamp(max=N - 1)
    qf = q[rows].float().view(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    L = table.shape[1] * c["page"]
    k = s["k"][table].permute(0, 2, 1, 3, 4).reshape(B, H, L, D).float()
    v = s["v"][table].permute(0, 2, 1, 3, 4).reshape(B, H, L, D).float()
    score = torch.matmul(qf, k.transpose(-1, -2)) * D ** -0.5
    pos = torch.arange(L, device=DEV)
    last = (s["len"].long() - n)[:, None] + torch.arange(R, device=DEV)
    seen = pos <= last[:, :, None]
    if c["window"]:
        seen = seen & (pos > last[:, :, None] - c["window"])
    seen = seen[:, None, :, None, :].expand(B, 1, R, G, L).reshape(B, 1, R * G, L)
    score = score.masked_fill(~seen, -math.inf)
    m = score.amax(-1, keepdim=True)
    e = (score - m).exp()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / total
    lse = (m + total.log())[..., 0]
    o = o.view(B, H, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, H * G, D)
    lse = lse.view(B, H, R, G).permute(0, 2, 1, 3).reshape(B, R, H * G)
    return [o[seq, i].to(q.dtype), lse[seq, i]]


# the cache in its plain form: a page is free where its count of users is 0; the lowest free pages are taken first

def _ceil(a, P):
    return (a + P - 1).div(P, rounding_mode="floor")


def _plain_reserve(s, seqs, num_new, total):
    """Extends each sequence by its new tokens; a shared, partly filled last page is copied first.  The new tokens' places."""
    P, at = s["case"]["page"], seqs.long()
    L, n = s["len"][at].long(), num_new.long()
    had = _ceil(L, P)
    tail = s["table"][at, (had - 1).clamp(min=0)].long()
    cow = (L % P > 0) & (n > 0) & (s["ref"][tail.clamp(min=0)] > 1)
    need = _ceil(L + n, P) - had + cow
    ends = need.cumsum(0)
    free = (s["ref"] == 0).nonzero()[:, 0]
    ok = (need == 0) | (ends <= free.numel())
    need = torch.where(ok, need, 0)
    owner = torch.repeat_interleave(torch.arange(at.numel(), device=DEV), need)
    page = free[:owner.numel()]
    j = torch.arange(owner.numel(), device=DEV) - (ends - need)[owner]
    col = (had - cow.long())[owner] + j
    s["ref"].scatter_add_(0, torch.where(cow & ok, tail, 0), -(cow & ok).to(torch.int32))
    s["ref"][page] = 1
    s["table"][at[owner], col] = page.to(torch.int32)
    copy = (cow & ok).nonzero()[:, 0]
    src, dst = tail[copy], s["table"][at[copy], had[copy] - 1].long()
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    s["len"][at] = (L + torch.where(ok, n, 0)).to(torch.int32)
    row = torch.repeat_interleave(torch.arange(at.numel(), device=DEV), n, output_size=total)
    where = L[row] + torch.arange(total, device=DEV) - (n.cumsum(0) - n)[row]
    return torch.where(ok[row], s["table"][at[row], where // P].long() * P + where % P, -1)


def _plain_drop(s, seqs, drop):
    """Takes the last tokens off each sequence, and the pages that no longer hold any of its tokens."""
    P, at = s["case"]["page"], seqs.long()
    L = s["len"][at].long()
    left = L - drop.long()
    col = torch.arange(s["table"].shape[1], device=DEV)
    gone = (col >= _ceil(left, P)[:, None]) & (col < _ceil(L, P)[:, None])
    rows = s["table"][at]
    s["ref"].scatter_add_(0, rows.clamp(min=0).long().view(-1), -gone.to(torch.int32).view(-1))
    s["table"][at] = torch.where(gone, -1, rows)
    s["len"][at] = left.to(torch.int32)


def _run_round(s):
    if own:
        c = s["cache"]
        c.truncate(s["seqs"], s["kept"])
        r = c.reserve(s["seqs"], s["num_new"], s["total"])
        for y in range(s["case"]["layers"]):
            c.write(y, s["k_new"][y], s["v_new"][y], r["slots"])
        c.commit(s["seqs"], s["num_draft"], s["accepted"])
        return [r["slots"], c.page_table, c.seq_len, c.refcount, c.k, c.v]
    P = s["case"]["page"]
    _plain_drop(s, s["seqs"], s["kept"])
    slots = _plain_reserve(s, s["seqs"], s["num_new"], s["total"])
    page, at = slots // P, slots % P
    s["k"][:, page, :, at] = s["k_new"].transpose(0, 1)
    s["v"][:, page, :, at] = s["v_new"].transpose(0, 1)
    _plain_drop(s, s["seqs"], s["num_draft"] - s["accepted"])
    return [slots, s["table"], s["len"], s["ref"], s["k"], s["v"]]


def _run_branch(s):
    if own:
        c = s["cache"]
        c.fork(s["parents"], s["children"])
        r = c.reserve(s["children"], s["num_new"], s["total"])
        held = c.page_table.clone()
        c.release(s["children"])
        return [r["slots"], held, c.page_table, c.seq_len, c.refcount, c.k, c.v]
    a, b = s["parents"].long(), s["children"].long()
    rows = s["table"][a]
    s["table"][b] = rows
    s["len"][b] = s["len"][a]
    s["ref"].scatter_add_(0, rows.clamp(min=0).long().view(-1), (rows >= 0).to(torch.int32).view(-1))
    slots = _plain_reserve(s, s["children"], s["num_new"], s["total"])
    held = s["table"].clone()
    _plain_drop(s, s["children"], s["len"][b])
    return [slots, held, s["table"], s["len"], s["ref"], s["k"], s["v"]]


def _run_compact(s):
    t = s["turn"]
    s["turn"] = 1 - t
    seqs, back, total = s["group%d" % t], s["back%d" % t], s["total%d" % t]
    if own:
        c = s["cache"]
        c.release(seqs)
        live = c.compact()
        slots = c.reserve(seqs, back, total)["slots"]
        return [live, slots, c.page_table, c.seq_len, c.refcount, c.k, c.v]
    _plain_drop(s, seqs, s["len"][seqs.long()])
    used = s["ref"] > 0
    live = used.sum().to(torch.int32).view(1)
    page = torch.arange(used.numel(), device=DEV)
    dst = ((page < live) & ~used).nonzero()[:, 0]
    src = ((page >= live) & used).nonzero()[:, 0]
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    s["ref"][dst] = s["ref"][src]
    s["ref"][src] = 0
    to = page.clone()
    to[src] = dst
    s["table"].copy_(torch.where(s["table"] < 0, -1, to[s["table"].clamp(min=0).long()].to(torch.int32)))
    slots = _plain_reserve(s, seqs, back, total)
    return [live, slots, s["table"], s["len"], s["ref"], s["k"], s["v"]]


# ---------------------------------------------------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"logprobs": _exact_logprobs, "attn": _exact_attn}.get(case["op"], _exact_cache)(case, s)


def _exact_logprobs(case, s):
    N, V, top = s["logits"].shape[0], case["vocab"], case["top"]
    tokens = s["tokens"].tolist()
    lp = torch.zeros(N, dtype=torch.float64, device=DEV)
    h, best = torch.zeros_like(lp), torch.full((N, top), -math.inf, dtype=torch.float64, device=DEV)
    for r in range(N):
        if tokens[r] < 0:
            continue
        x = s["logits"][r, :V].double()
        if s["temperature"] is not None:
            x = x / s["temperature"][r].double()
        logp = x - torch.logsumexp(x, 0)
        lp[r] = logp[tokens[r]]
        h[r] = -(logp.exp() * logp).sum()
        best[r] = logp.sort(descending=True).values[:top]
    return [lp, h, None, None, best]


def _exact_attn(case, s):
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    G = case["heads"] // H
    out, lse, row = [], [], 0
    for b, (length, drafts) in enumerate(zip(s["len"].tolist(), s["num_draft"].tolist())):
        pages = s["table"][b, :-(-length // P)].long()
        k = s["k"][pages].transpose(0, 1).reshape(H, -1, D)[:, :length].double()
        v = s["v"][pages].transpose(0, 1).reshape(H, -1, D)[:, :length].double()
        for i in range(drafts + 1):
            end = length - drafts + i
            start = max(0, end - case["window"]) if case["window"] else 0
            q = s["q"][row].double().view(H, G, D)
            score = torch.matmul(q, k[:, start:end].transpose(1, 2).contiguous()) / math.sqrt(D)
            out.append(torch.matmul(torch.softmax(score, -1), v[:, start:end].contiguous()).view(H * G, D))
            lse.append(torch.logsumexp(score, -1).view(H * G))
            row += 1
    return [torch.stack(out), torch.stack(lse)]


class _Book:
    """The cache's bookkeeping with Python lists, one sequence after the other."""

    def __init__(self, s, P):
        self.P, self.k, self.v = P, s["k"].double(), s["v"].double()
        self.len, self.ref = s["len"].tolist(), s["ref"].tolist()
        self.pages = [[p for p in row if p >= 0] for row in s["table"].tolist()]

    def reserve(self, seqs, new):
        free = [p for p, r in enumerate(self.ref) if r == 0][::-1]
        before, places, copies = list(self.ref), [], []
        for b, n in zip(seqs, new):
            if n and self.len[b] % self.P and before[self.pages[b][-1]] > 1:
                old, self.pages[b][-1] = self.pages[b][-1], free.pop()
                self.ref[old] -= 1
                self.ref[self.pages[b][-1]] = 1
                copies.append((old, self.pages[b][-1]))
            for _ in range(n):
                if self.len[b] == len(self.pages[b]) * self.P:
                    self.pages[b].append(free.pop())
                    self.ref[self.pages[b][-1]] = 1
                places.append((self.pages[b][self.len[b] // self.P], self.len[b] % self.P))
                self.len[b] += 1
        self.move(copies)
        return places

    def move(self, pairs):
        if pairs:
            a, b = (torch.tensor(x, device=DEV) for x in zip(*pairs))
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]

    def drop(self, b, n):
        self.len[b] -= n
        while len(self.pages[b]) > -(-self.len[b] // self.P):
            self.ref[self.pages[b].pop()] -= 1


def _exact_cache(case, s):
    """The pool after the pass (the whole numbers are held to equality with the plain form's)."""
    book, op = _Book(s, case["page"]), case["op"]
    if op == "round":
        seqs = s["seqs"].tolist()
        for b, n in zip(seqs, s["kept"].tolist()):
            book.drop(b, n)
        page, at = (torch.tensor(x, device=DEV) for x in zip(*book.reserve(seqs, s["num_new"].tolist())))
        book.k[:, page, :, at] = s["k_new"].double().transpose(0, 1)
        book.v[:, page, :, at] = s["v_new"].double().transpose(0, 1)
        return [None, None, None, None, book.k, book.v]
    if op == "branch":
        for a, b in zip(s["parents"].tolist(), s["children"].tolist()):
            book.pages[b], book.len[b] = list(book.pages[a]), book.len[a]
            for p in book.pages[a]:
                book.ref[p] += 1
        book.reserve(s["children"].tolist(), s["num_new"].tolist())
        return [None, None, None, None, None, book.k, book.v]
    for b in s["group0"].tolist():
        book.drop(b, book.len[b])
    used = [p for p, r in enumerate(book.ref) if r]
    holes = [p for p in range(len(used)) if not book.ref[p]]
    book.move(list(zip([p for p in used if p >= len(used)], holes)))
    return [None, None, None, None, None, book.k, book.v]
