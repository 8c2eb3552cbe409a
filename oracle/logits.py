"""Penalties, biases and masks on rows of logits, plain fp64 -- TEST INFRASTRUCTURE (same rules as the rest of
``oracle/``).

Page: "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.1: candidates of a step are selected from the
next-token logits.  The rules are those that the header states for ``bg_adjust_logits``, applied token by token.
"""
from __future__ import annotations

import numpy as np


def adjust(logits, per, prompts=None, own=None, repetition=None, frequency=None, presence=None, biases=None, masks=None):
    """logits [N,V]; per group: prompts (lists of tokens), repetition, frequency, presence, biases (lists of (token,
    value)); per row: own (lists of tokens), masks (sets of allowed tokens, or None).  Returns (out, size): size is the
    sum of the magnitudes that an element passed through."""
    x = np.asarray(logits, dtype=np.float64)
    N, V = x.shape
    out, size = x.copy(), np.abs(x)
    for i in range(N):
        g = i // per
        counts = {}
        for t in (own[i] if own is not None else ()):
            if 0 <= t < V:
                counts[t] = counts.get(t, 0) + 1
        touched = set(counts) | {t for t in (prompts[g] if prompts is not None else ()) if 0 <= t < V}
        if repetition is not None:
            r = float(repetition[g])
            for t in touched:
                out[i, t] = out[i, t] / r if out[i, t] > 0 else out[i, t] * r
                size[i, t] = abs(out[i, t])
        a = 0.0 if frequency is None else float(frequency[g])
        b = 0.0 if presence is None else float(presence[g])
        for t, c in counts.items():
            out[i, t] -= a * c + b
            size[i, t] += abs(a * c) + abs(b)
        for t, v in dict(biases[g] if biases is not None else ()).items():
            if 0 <= t < V:
                out[i, t] += float(v)
                size[i, t] += abs(float(v))
        if masks is not None and masks[i] is not None:
            banned = np.ones(V, bool)
            banned[[t for t in masks[i] if t < V]] = False
            out[i, banned] = -np.inf
    return out, size
