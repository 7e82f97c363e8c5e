"""Log probabilities, entropy, rank and top alternatives of rows of logits (oracle, test infrastructure).

Graft article, architecture paragraph: the emitted tokens follow the target's
own distribution, p = softmax(logits / T).  In float64 from the definitions:
log p = z - log sum exp z, H = -sum p log p, alternatives by (logit
descending, id ascending) with NaN as low as -inf, rank = a token's place
among them.
"""
from __future__ import annotations

import numpy as np


def row(x, token: int, top: int, T: float = 1.0):
    """x [V]; returns (log p of token or 0 without one, entropy, rank or -1, ids [top], their log p)."""
    x = np.asarray(x, np.float64)
    lawful = not np.isnan(x).any() and not (x == np.inf).any() and (x > -np.inf).any()
    if lawful:
        z = x / T
        z = z - z.max()
        logp = z - np.log(np.exp(z).sum())
        p = np.exp(logp)
        entropy = -(p[p > 0] * logp[p > 0]).sum()
    else:
        logp, entropy = np.full(len(x), np.nan), np.nan
    order = np.argsort(np.where(np.isnan(x), np.inf, -x), kind="stable")
    rank = int(np.flatnonzero(order == token)[0]) if token >= 0 else -1
    return (logp[token] if token >= 0 else 0.0), entropy, rank, order[:top], logp[order[:top]]


def tokens(logits, toks, rows=None, block: int = 0, top: int = 0, T: float = 1.0):
    """graft_token_logprobs: logits [R][V], toks [N], rows [N] or None."""
    n = len(toks)
    out = dict(logprob=np.zeros(n), entropy=np.zeros(n), rank=np.full(n, -1), top_id=np.full((n, top), -1),
               top_logprob=np.zeros((n, top)))
    for i in range(n):
        r = i if rows is None else int(rows[i])
        if r < 0:
            continue
        r += i // block * block if block else 0
        (out["logprob"][i], out["entropy"][i], out["rank"][i], out["top_id"][i],
         out["top_logprob"][i]) = row(logits[r], int(toks[i]), top, T)
    return out
