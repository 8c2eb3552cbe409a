"""Norm of the heads of Q and K and their rotation by position, plain fp64 numpy -- TEST INFRASTRUCTURE
(same rules as the rest of ``oracle/``).

Page: "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.2: the attention works on packed
tokens whose K is kept rotated.  A head x of a token becomes y = x / sqrt(mean(x^2) + eps) * (offset + w), and
each pair (a, b) of its first 2 n dimensions is turned as the complex number y_a + i y_b by
scale * exp(i * position[axis] * frequency).
"""
from __future__ import annotations

import numpy as np


def norm_rotate(x, weight, eps, offset, pos, inv_freq, axis_of=None, interleaved=False, scale=1.0):
    """x [rows,H,d], pos [axes,rows], inv_freq [n].  Returns (out, size): out [rows,H,d] and what its elements are
    made of, |y_a| + |y_b| of their pair (|y| where nothing turns)."""
    x = np.asarray(x, dtype=np.float64)
    y = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (offset + np.asarray(weight))
    n = len(inv_freq)
    out, size = y.copy(), np.abs(y)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        angle = np.asarray(pos[0 if axis_of is None else axis_of[i]], dtype=np.float64) * float(inv_freq[i])
        z = (y[..., a] + 1j * y[..., b]) * (scale * np.exp(1j * angle))[:, None]
        out[..., a], out[..., b] = z.real, z.imag
        size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, size
