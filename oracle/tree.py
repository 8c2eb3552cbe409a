"""Attention of drafted trees over their request's prefix, plain fp64 numpy -- TEST INFRASTRUCTURE (same rules as
the rest of ``oracle/``).

Page: "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.2: what sequences of a request share is kept
once.  A node of a tree stands for the sequence [prefix ; path from the root to it]; its attention is the last row
of that sequence's.
"""
from __future__ import annotations

import numpy as np


def path(parent, i):
    """Node i and its ancestors, from the root on; a parent that is no lower node ends the path."""
    nodes = [i]
    while 0 <= parent[nodes[-1]] < nodes[-1]:
        nodes.append(int(parent[nodes[-1]]))
    return nodes[::-1]


def attn(q, k, v, parent, cu_nodes, prefix_k, prefix_v, cu_prefix, scale, softcap=0.0):
    """fp64 arrays q [T,Hq,d], k/v [T,Hkv,d], prefix_k/v [P,Hkv,d], parent [T] within its request.  Returns
    (out, lse, mean_abs, dot_abs) as ``shared.attn`` does."""
    T, Hq, d = q.shape
    g = Hq // k.shape[1]
    out, mean_abs = np.empty((T, Hq, d)), np.empty((T, Hq, d))
    lse, dot_abs = np.empty((T, Hq)), np.empty((T, Hq))
    for r in range(len(cu_nodes) - 1):
        a, b = int(cu_nodes[r]), int(cu_nodes[r + 1])
        pk, pv = prefix_k[cu_prefix[r]:cu_prefix[r + 1]], prefix_v[cu_prefix[r]:cu_prefix[r + 1]]
        for i in range(b - a):
            rows = [a + n for n in path(parent[a:b], i)]
            keys, vals = np.concatenate((pk, k[rows])), np.concatenate((pv, v[rows]))
            for h in range(Hq):
                kk, qq = keys[:, h // g], q[a + i, h]
                x = scale * (kk @ qq)
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                w = np.exp(x - x.max())
                out[a + i, h] = (w / w.sum()) @ vals[:, h // g]
                mean_abs[a + i, h] = (w / w.sum()) @ np.abs(vals[:, h // g])
                lse[a + i, h] = x.max() + np.log(w.sum())
                dot_abs[a + i, h] = (scale * (np.abs(kk) @ np.abs(qq))).max()
    return out, lse, mean_abs, dot_abs
