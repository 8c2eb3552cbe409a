"""Log-probabilities, entropy and best alternatives of rows of logits, plain fp64 numpy -- TEST
INFRASTRUCTURE (same rules as the rest of ``oracle/``).

Page: "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.1: a Prefill-Only request is
answered from the softmax of the next-token logits at the last valid position, or its Top-K.
Equal logits are ordered by the smaller token; 0 log 0 = 0.
"""
from __future__ import annotations

import numpy as np


def token_logprobs(logits, tokens, K):
    """logits [N,V]; returns fp64 logprob [N], entropy [N], int64 top_token [N,K], top_logprob [N,K]."""
    x = np.asarray(logits, dtype=np.float64)
    N = x.shape[0]
    lp, H = np.empty(N), np.empty(N)
    top, tlp = np.empty((N, K), np.int64), np.empty((N, K))
    for i in range(N):
        row = x[i]
        if np.isnan(row).any() or np.isposinf(row).any():
            lp[i], H[i], top[i], tlp[i] = np.nan, np.nan, -1, np.nan
            continue
        order = np.lexsort((np.arange(row.size), -row))[:K]
        top[i] = order
        m = row.max()
        if m == -np.inf:
            lp[i], H[i], tlp[i] = -np.inf, 0.0, -np.inf
            continue
        # relative to the maximum throughout: m + log(sum) would lose the sum next to a huge m
        logp = (row - m) - np.log(np.exp(row - m).sum())
        p = np.exp(logp)
        H[i] = -(p[p > 0] * logp[p > 0]).sum()
        lp[i] = logp[tokens[i]]
        tlp[i] = logp[order]
    return lp, H, top, tlp
