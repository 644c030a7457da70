"""Log probabilities of given tokens, ranks, entropy and top alternatives, in float64."""
import numpy as np


def token_logprobs(logits, token_ids, top_k):
    """``logits`` [rows, vocab] float64 -> (logprobs, ranks, entropy, top_ids, top_logprobs).

    A row with NaN or +inf has no distribution (NaN, rank 0, ids -1); a row of nothing but -inf
    has log probabilities -inf and entropy 0; token id -1 asks for none (0, rank 0)."""
    rows, vocab = logits.shape
    lp = np.zeros(rows)
    rank = np.zeros(rows, np.int32)
    ent = np.zeros(rows)
    ids = np.full((rows, top_k), -1, np.int32)
    best = np.full((rows, top_k), -np.inf)
    for r in range(rows):
        x = logits[r]
        t = int(token_ids[r])
        if np.isnan(x).any() or (x == np.inf).any():
            lp[r] = ent[r] = np.nan
            best[r] = np.nan
            continue
        m = x.max()
        if m == -np.inf:
            p, logp = np.zeros(vocab), np.full(vocab, -np.inf)
        else:
            with np.errstate(under="ignore"):
                z = np.exp(x - m).sum()
                logp = (x - m) - np.log(z)
                p = np.exp(logp)
        ent[r] = -(p[p > 0] * logp[p > 0]).sum()
        if t >= 0:
            lp[r] = logp[t]
            rank[r] = 1 + int((x > x[t]).sum())
        order = np.lexsort((np.arange(vocab), -x))[:top_k]
        ids[r, :order.size] = order
        best[r, :order.size] = logp[order]
    return lp, rank, ent, ids, best
