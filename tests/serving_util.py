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
