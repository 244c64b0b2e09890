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


class CacheModel:
    """The paged cache with Python lists and one token's (k, v) per place:
    sequence by sequence, page by page."""

    def __init__(self, c):
        self.P, self.W, self.NP = c.page_size, c.page_table.shape[1], c.refcount.shape[0]
        self.len = [0] * c.seq_len.shape[0]
        self.pages = [[] for _ in self.len]
        self.ref = [0] * self.NP
        self.k, self.v = c.k.cpu().clone(), c.v.cpu().clone()

    def _slots(self, seqs):
        seen = set()
        for s in seqs:
            yield s, 0 <= s < len(self.len) and s not in seen
            seen.add(s)

    def reserve(self, seqs, new, total):
        if any(n < 0 for n in new) or sum(new) != total:
            return [-1] * len(seqs), [-1] * total, [1] * len(seqs)
        before, start, slots, status, moves = list(self.ref), [], [], [], []
        free = [p for p in range(self.NP) if before[p] == 0]
        asked = 0
        for (s, ok), n in zip(self._slots(seqs), new):
            st = 0 if ok else 256
            if ok and self.len[s] + n > self.W * self.P:
                st = 512
            if not st:
                L = self.len[s]
                cow = n > 0 and L % self.P > 0 and before[self.pages[s][-1]] > 1
                need = -(-(L + n) // self.P) - len(self.pages[s]) + cow
                asked += need
                if need and asked > len(free):
                    st = 2048
            if st:
                start.append(-1)
                slots += [-1] * n
            else:
                take = free[asked - need:asked]
                if cow:
                    old = self.pages[s][-1]
                    self.ref[old] -= 1
                    self.pages[s][-1] = take[0]
                    moves.append((old, take[0]))
                self.pages[s] += take[cow:]
                for p in take:
                    self.ref[p] = 1
                self.len[s] = L + n
                start.append(L)
                slots += [self.pages[s][j // self.P] * self.P + j % self.P for j in range(L, L + n)]
            status.append(st)
        self._move(moves)
        return start, slots, status

    def _move(self, moves):
        if moves:
            a, b = (torch.tensor(x) for x in zip(*moves))
            self.k[:, b], self.v[:, b] = self.k[:, a].clone(), self.v[:, a].clone()

    def write(self, layer, k, v, slots):
        for r, s in enumerate(slots):
            if s >= 0:
                self.k[layer, s // self.P, :, s % self.P] = k[r]
                self.v[layer, s // self.P, :, s % self.P] = v[r]

    def truncate(self, seqs, drop):
        status = []
        for (s, ok), d in zip(self._slots(seqs), drop):
            st = 256 if not ok else 512 if d is None or not 0 <= d <= self.len[s] else 0
            if not st:
                self.len[s] -= d
                while len(self.pages[s]) > -(-self.len[s] // self.P):
                    self.ref[self.pages[s].pop()] -= 1
            status.append(st)
        return status

    def commit(self, seqs, K, A):
        return self.truncate(seqs, [k - a if k >= 0 and -1 <= a <= k else None for k, a in zip(K, A)])

    def release(self, seqs):
        return self.truncate(seqs, [self.len[s] if 0 <= s < len(self.len) else 0 for s in seqs])

    def fork(self, parents, children):
        was = list(self.len)
        status = []
        for p, (c, ok) in zip(parents, list(self._slots(children))):
            st = 256 if not ok or not 0 <= p < len(was) else 512 if was[c] else 0
            if not st and was[p]:
                self.len[c], self.pages[c] = was[p], list(self.pages[p])
                for q in self.pages[p]:
                    self.ref[q] += 1
            status.append(st)
        return status

    def compact(self):
        used = [p for p in range(self.NP) if self.ref[p]]
        holes = [p for p in range(len(used)) if not self.ref[p]]
        movers = [p for p in used if p >= len(used)]
        self._move(list(zip(movers, holes)))
        name = dict(zip(movers, holes))
        for p, h in name.items():
            self.ref[h], self.ref[p] = self.ref[p], 0
        self.pages = [[name.get(p, p) for p in row] for row in self.pages]
        return len(used)

    def check(self, c):
        assert c.seq_len.tolist() == self.len
        assert c.refcount.tolist() == self.ref
        want = [row + [-1] * (self.W - len(row)) for row in self.pages]
        assert c.page_table.tolist() == want
        assert torch.equal(c.k.cpu().view(torch.int16), self.k.view(torch.int16))
        assert torch.equal(c.v.cpu().view(torch.int16), self.v.view(torch.int16))
