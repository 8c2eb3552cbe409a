"""Attention of a request's samples over its one prefix, plain fp64 numpy -- TEST INFRASTRUCTURE.

Same rules as the rest of ``oracle/``: only ``tests/`` and ``__graft_entry__.smoke()`` may use it;
it never imports the product.

Page: "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", abstract and section 1.2: a Prefill-Only
request carries several samples, and state its sequences share is kept once per request.  Reading:
sample s of request r is the sequence [prefix of r ; s], so its tokens attend to the whole prefix
and, causally, to their own sample; the last-token form is the row of the sequence's end.  Capped
scores are cap * tanh(x / cap) of the scaled products x.
"""
from __future__ import annotations

import numpy as np


def attn(q, k, v, cu, prefix_k, prefix_v, cu_prefix, cu_group, scale, softcap=0.0, last=False):
    """fp64 arrays q [rows,Hq,d], k/v [T,Hkv,d], prefix_k/v [P,Hkv,d].  Returns (out, lse, mean_abs, dot_abs):
    out [rows,Hq,d] (NaN for a query without keys), lse [rows,Hq], the weighted mean of |v|
    [rows,Hq,d] and the largest scale * sum |q_i k_i| over the keys of a query [rows,Hq]."""
    rows, Hq, d = q.shape
    Hkv = k.shape[1] if k.shape[0] else prefix_k.shape[1]
    g = Hq // Hkv
    out = np.full((rows, Hq, d), np.nan)
    mean_abs = np.zeros((rows, Hq, d))
    lse = np.full((rows, Hq), -np.inf)
    dot_abs = np.zeros((rows, Hq))
    for r in range(len(cu_group) - 1):
        pk = prefix_k[cu_prefix[r]:cu_prefix[r + 1]]
        pv = prefix_v[cu_prefix[r]:cu_prefix[r + 1]]
        for s in range(cu_group[r], cu_group[r + 1]):
            a, b = int(cu[s]), int(cu[s + 1])
            keys = np.concatenate((pk, k[a:b]))
            vals = np.concatenate((pv, v[a:b]))
            queries = [(s, len(keys))] if last else [(t, len(pk) + t - a + 1) for t in range(a, b)]
            for row, n in queries:
                if n == 0:
                    continue
                for kh in range(Hkv):
                    qq = q[row, kh * g:(kh + 1) * g]                       # [g, d]
                    x = scale * (qq @ keys[:n, kh].T)                      # [g, n]
                    if softcap:
                        x = softcap * np.tanh(x / softcap)
                    top = x.max(axis=1, keepdims=True)
                    w = np.exp(x - top)
                    z = w.sum(axis=1, keepdims=True)
                    h = slice(kh * g, (kh + 1) * g)
                    out[row, h] = (w / z) @ vals[:n, kh]
                    mean_abs[row, h] = (w / z) @ np.abs(vals[:n, kh])
                    lse[row, h] = (top + np.log(z))[:, 0]
                    dot_abs[row, h] = (scale * (np.abs(qq) @ np.abs(keys[:n, kh]).T)).max(axis=1)
    return out, lse, mean_abs, dot_abs
