"""Pins of the shared-prefix oracle (oracle/shared.py) to things other than itself: the packed
prefill and last-token oracles over materialised [prefix ; sample] sequences, closed forms of the
capped score, and the equality of the two forms on a sample's last row."""
import math

import numpy as np

import oracle
from attention_packed_varlen_causal_gb300 import workloads as wl
from oracle import shared as sh


def problem(seed, prefix, groups, Hq=4, Hkv=2, d=64):
    rng = np.random.default_rng(seed)
    lens = [n for g in groups for n in g]
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    cup = np.concatenate(([0], np.cumsum(prefix))).astype(np.int32)
    cug = np.concatenate(([0], np.cumsum([len(g) for g in groups]))).astype(np.int32)
    bits = {n: wl.bf16_bits_from_f32(rng.standard_normal(s, dtype=np.float32)) for n, s in
            dict(q=(cu[-1], Hq, d), k=(cu[-1], Hkv, d), v=(cu[-1], Hkv, d), pk=(cup[-1], Hkv, d), pv=(cup[-1], Hkv, d),
                 pq=(cup[-1], Hq, d)).items()}
    return bits, cu, cup, cug


def f64(b):
    return wl.bf16_bits_to_f32(b).astype(np.float64)


def test_equals_prefill_of_materialised_sequences():
    x, cu, cup, cug = problem(5, [7, 0, 12], [[3, 1, 5], [4], [2, 6]])
    out, _, _, _ = sh.attn(f64(x["q"]), f64(x["k"]), f64(x["v"]), cu, f64(x["pk"]), f64(x["pv"]), cup, cug, 0.125)
    for r in range(3):
        p = slice(cup[r], cup[r + 1])
        for s in range(cug[r], cug[r + 1]):
            own = slice(cu[s], cu[s + 1])
            cat = {n: np.concatenate((x[a][p], x[b][own])) for n, a, b in (("q", "pq", "q"), ("k", "pk", "k"),
                                                                            ("v", "pv", "v"))}
            L = cat["q"].shape[0]
            ref = oracle.prefill(cat["q"], cat["k"], cat["v"], np.array([0, L], np.int32), 0.125)
            ref = ref[0] if isinstance(ref, tuple) else ref
            assert np.allclose(out[own], ref[L - (cu[s + 1] - cu[s]):], rtol=0, atol=1e-12)


def test_last_token_is_the_prefill_row_of_the_sample_end():
    x, cu, cup, cug = problem(6, [9, 3], [[3, 1], [4, 2, 8]])
    args = (f64(x["k"]), f64(x["v"]), cu, f64(x["pk"]), f64(x["pv"]), cup, cug, 0.2)
    for cap in (0.0, 1.5):
        full, lse, _, _ = sh.attn(f64(x["q"]), *args, softcap=cap)
        ends = cu[1:] - 1
        one, lse1, _, _ = sh.attn(f64(x["q"])[ends], *args, softcap=cap, last=True)
        assert np.allclose(one, full[ends], rtol=0, atol=1e-14) and np.allclose(lse1, lse[ends], rtol=0, atol=1e-14)


def test_two_keys_closed_form_with_cap():
    # one head, d 64, q = e0, keys a e0 and b e0: weights by the logistic function of the capped difference
    q = np.zeros((1, 1, 64)); q[0, 0, 0] = 1.0
    k = np.zeros((1, 1, 64)); k[0, 0, 0] = 3.0
    pk = np.zeros((1, 1, 64)); pk[0, 0, 0] = -2.0
    v = np.full((1, 1, 64), 1.0)
    pv = np.full((1, 1, 64), 5.0)
    for cap in (0.0, 0.7, 40.0):
        f = (lambda t: cap * math.tanh(t / cap)) if cap else (lambda t: t)
        w = 1.0 / (1.0 + math.exp(f(-2.0) - f(3.0)))          # weight of the own key
        out, lse, _, _ = sh.attn(q, k, v, [0, 1], pk, pv, [0, 1], [0, 1], 1.0, softcap=cap)
        assert np.allclose(out, w * 1.0 + (1 - w) * 5.0, rtol=0, atol=1e-13)
        assert abs(lse[0, 0] - math.log(math.exp(f(-2.0)) + math.exp(f(3.0)))) < 1e-13


def test_query_without_keys():
    x, cu, cup, cug = problem(7, [0, 2], [[0, 2], [0]])
    out, lse, _, _ = sh.attn(np.ones((3, 4, 64)), f64(x["k"]), f64(x["v"]), cu, f64(x["pk"]), f64(x["pv"]), cup, cug,
                             0.1, last=True)
    assert np.isnan(out[0]).all() and np.isfinite(out[1:]).all() and np.all(lse[0] == -np.inf)
