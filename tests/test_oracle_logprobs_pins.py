"""Pins of the log-probability oracle (oracle/logprobs.py) to closed forms and brute force."""
import math

import numpy as np

from oracle import logprobs as ol


def test_two_tokens_closed_form():
    a, b = 0.7, -1.9
    lp, H, top, tlp = ol.token_logprobs([[a, b], [b, a]], [0, 0], 2)
    p = 1 / (1 + math.exp(b - a))
    h = -p * math.log(p) - (1 - p) * math.log(1 - p)
    assert np.allclose(lp, [math.log(p), math.log(1 - p)], atol=1e-14) and np.allclose(H, h, atol=1e-14)
    assert top.tolist() == [[0, 1], [1, 0]]
    assert np.allclose(tlp, [math.log(p), math.log(1 - p)], atol=1e-14)


def test_uniform_rows_and_ties():
    lp, H, top, _ = ol.token_logprobs(np.full((1, 50), 3.0), [17], 4)
    assert np.allclose(lp, -math.log(50)) and np.allclose(H, math.log(50)) and top.tolist() == [[0, 1, 2, 3]]


def test_uniform_rows_at_the_types_ends():
    for x in (-3.4e38, 3.4e38):
        lp, H, _, tlp = ol.token_logprobs(np.full((1, 50), x), [17], 1)
        assert np.allclose([lp[0], -H[0], tlp[0, 0]], -math.log(50))


def test_shift_invariance_and_bans():
    x = np.random.default_rng(3).normal(0, 2, (3, 40))
    x[:, ::3] = -np.inf
    a, b = ol.token_logprobs(x, [1, 2, 4], 30), ol.token_logprobs(x + 100.0, [1, 2, 4], 30)
    for u, v in zip(a, b):
        assert np.allclose(np.where(np.isfinite(u), u, 0), np.where(np.isfinite(v), v, 0), atol=1e-11)
    live = [v for v in range(40) if v % 3]
    p = np.exp(x[0, live]) / np.exp(x[0, live]).sum()
    assert np.allclose(a[1][0], -(p * np.log(p)).sum())
    assert a[2][0].tolist()[26:] == [0, 3, 6, 9]          # 26 live tokens, then the banned ones in order


def test_rows_without_a_distribution():
    x = np.zeros((3, 5))
    x[0] = -np.inf
    x[1, 2] = np.nan
    x[2, 1] = np.inf
    lp, H, top, tlp = ol.token_logprobs(x, [0, 0, 0], 2)
    assert lp[0] == -np.inf and H[0] == 0 and top[0].tolist() == [0, 1] and (tlp[0] == -np.inf).all()
    assert np.isnan(lp[1:]).all() and np.isnan(H[1:]).all() and (top[1:] == -1).all()
