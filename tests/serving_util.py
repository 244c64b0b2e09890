"""Plain float64 forms of the serving operators, for their tests."""
import numpy as np
import torch


def logprobs_ref(logits, tokens, temperature, vocab, top):
    """Row by row in float64 on the CPU: logprob, entropy, rank, top tokens
    (value descending, index ascending) and their log probabilities."""
    x_all = logits.detach().cpu().to(torch.float64).numpy()[:, :vocab]
    R = x_all.shape[0]
    lp, ent, rank = np.zeros(R), np.zeros(R), np.zeros(R, np.int64)
    ids, tlp = np.full((R, top), -1, np.int64), np.full((R, top), -np.inf)
    for r in range(R):
        t = None if tokens is None else int(tokens[r])
        if t is not None and t < 0:
            continue
        raw = x_all[r]
        x = raw / (1.0 if temperature is None else float(temperature[r]))
        y = x - x.max()
        e = np.exp(y)
        s = e.sum()
        logp = y - np.log(s)
        seen = e > 0
        ent[r] = np.log(s) - (e[seen] * y[seen]).sum() / s
        if t is not None:
            lp[r], rank[r] = logp[t], (raw > raw[t]).sum() + 1
        ids[r] = np.lexsort((np.arange(vocab), -raw))[:top]
        tlp[r] = logp[ids[r]]
    return dict(logprob=lp, entropy=ent, rank=rank, top_tokens=ids, top_logprobs=tlp)


def attention_ref(q, k, v, table, seq_len, num_draft, seqs=None, scale=None, window=0):
    """Row by row in float64 on the CPU, reading only visible positions."""
    q, k, v = (t.detach().cpu().to(torch.float64) for t in (q, k, v))
    table, seq_len, num_draft = table.cpu().numpy(), seq_len.cpu().numpy(), num_draft.cpu().numpy()
    N, H, D = q.shape
    KV, P = k.shape[1], k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, lse = torch.zeros(N, H, D, dtype=torch.float64), torch.full((N, H), -torch.inf, dtype=torch.float64)
    row = 0
    for b, nd in enumerate(num_draft):
        slot = b if seqs is None else int(seqs[b])
        L = int(seq_len[slot])
        pos = torch.arange(L)
        pages = torch.from_numpy(table[slot].astype(np.int64))[pos // P]
        kb, vb = k[pages, :, pos % P], v[pages, :, pos % P]            # [L, KV, D]
        for i in range(nd + 1):
            end = L - nd + i                                           # first position not seen
            start = max(0, end - window) if window else 0
            if end > start:
                kk = kb[start:end].repeat_interleave(H // KV, 1)
                vv = vb[start:end].repeat_interleave(H // KV, 1)
                s = (q[row][None] * kk).sum(-1) * scale                # [L, H]
                m = s.max(0).values
                e = (s - m).exp()
                out[row] = (e[:, :, None] * vv).sum(0) / e.sum(0)[:, None]
                lse[row] = m + e.sum(0).log()
            row += 1
    return out, lse


def make_pages(L, P, KV, D, dtype, seed, layout="head", extra=3):
    """Random pages in random order for sequences of the given lengths; what
    no token fills holds NaN.  layout "token": tokens before heads in memory."""
    g = torch.Generator().manual_seed(seed)
    n = [-(-x // P) for x in L]
    total = sum(n) + extra
    k, v = (torch.randn(total, KV, P, D, generator=g).to(dtype) for _ in range(2))
    ids = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(L), max(max(n), 1)), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(L):
        table[b, :n[b]] = ids[at:at + n[b]]
        if x % P:
            k[ids[at + n[b] - 1].long(), :, x % P:] = torch.nan
            v[ids[at + n[b] - 1].long(), :, x % P:] = torch.nan
        at += n[b]
    for p in ids[at:]:
        k[p.long()], v[p.long()] = torch.nan, torch.nan
    if layout == "token":
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))

    def up(t):
        return t.cuda() if t.is_contiguous() else t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    return up(k), up(v), table.cuda(), torch.tensor(L, dtype=torch.int32).cuda()
