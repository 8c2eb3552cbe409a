"""Pins of the oracles of the calls around a decode or verify step: norm and rotation, logit adjustments, trees."""
import math

import numpy as np
import pytest

from oracle import logits as olg
from oracle import rope as orp
from oracle import shared as osh
from oracle import tree as otr


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("interleaved", [False, True])
def test_quarter_turn(interleaved):
    """A position times frequency of pi / 2 takes (1, 0) to (0, 1)."""
    x = np.zeros((1, 1, 4))
    x[0, 0, 0] = 1
    out, _ = orp.norm_rotate(x, None, 0, 0, [[1]], [math.pi / 2, 0.0], interleaved=interleaved)
    want = np.zeros(4)
    want[1 if interleaved else 2] = 1
    assert np.allclose(out[0, 0], want, atol=1e-15)


def test_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    f = 10000.0 ** (-np.arange(8) / 8)

    def score(p, q):
        a, _ = orp.norm_rotate(x, None, 0, 0, [[p]], f)
        b, _ = orp.norm_rotate(y, None, 0, 0, [[q]], f)
        return (a * b).sum()

    x, y = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))
    assert abs(score(5, 3) - score(105, 103)) < 1e-12 and abs(score(5, 3) - score(5, 4)) > 1e-3


def test_norm_and_axes():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    out, _ = orp.norm_rotate(x, [1.0, 2.0, 1.0, 1.0], 0.0, 0.0, [[0]], [1.0])
    assert np.allclose(out, [[[1.2, 3.2, 0, 0]]])            # root mean square 2.5
    out, _ = orp.norm_rotate(x, np.zeros(4), 0.0, 1.0, [[0]], [1.0])
    assert np.allclose(out, x / 2.5)
    # two axes: each pair turns by its own position, the rest stays
    x = np.array([[[1.0, 1.0, 0.0, 0.0, 7.0, 8.0]]])
    out, size = orp.norm_rotate(x, None, 0, 0, [[0], [1]], [math.pi, math.pi / 2], axis_of=[0, 1])
    assert np.allclose(out, [[[1, 0, 0, 1, 7, 8]]]) and np.allclose(size, [[[1, 1, 1, 1, 7, 8]]])


# ------------------------------------------------------------------ logits
def test_logit_rules_by_hand():
    x = [[2.0, -2.0, 1.0, 0.5, 0.25]]
    out, _ = olg.adjust(x, 1, prompts=[[0, 1]], own=[[2, 2, 1]], repetition=[2.0], frequency=[0.25], presence=[0.5],
                        biases=[[(3, 9.0), (3, -1.0), (0, 1.0)]], masks=[{0, 1, 2, 3}])
    assert out.tolist() == [[2.0, -4.75, -0.5, -0.5, -math.inf]]


def test_logit_rules_one_at_a_time():
    x = np.array([[1.0, -1.0], [3.0, 4.0]])
    same, _ = olg.adjust(x, 2)
    assert (same == x).all()
    out, _ = olg.adjust(x, 1, own=[[], [1]], presence=[1.0, 1.0])
    assert out.tolist() == [[1, -1], [3, 3]]
    out, _ = olg.adjust(x, 2, masks=[set(), None])
    assert out.tolist() == [[-math.inf, -math.inf], [3, 4]]
    out, _ = olg.adjust(x, 2, prompts=[[-1, 5]], own=[[2], [-3]], repetition=[2.0])       # none of them a token
    assert (out == x).all()


# ------------------------------------------------------------------ trees
def make(seed, n, p, Hq=4, Hkv=2, d=8):
    rng = np.random.default_rng(seed)
    return [rng.normal(size=(m, h, d)) for m, h in ((n, Hq), (n, Hkv), (n, Hkv), (p, Hkv), (p, Hkv))]


def test_a_chain_is_a_causal_sample():
    q, k, v, pk, pv = make(1, 9, 5)
    cu, cup = [0, 4, 9], [0, 0, 5]
    parent = np.array([-1, 0, 1, 2, -1, 0, 1, 2, 3])
    got = otr.attn(q, k, v, parent, cu, pk, pv, cup, 0.3, softcap=2.0)
    want = osh.attn(q, k, v, cu, pk, pv, cup, [0, 1, 2], 0.3, softcap=2.0)
    for a, b in zip(got, want):
        assert np.allclose(a, b, atol=1e-12)


def test_roots_are_samples_of_one_token():
    q, k, v, pk, pv = make(2, 6, 7)
    got = otr.attn(q, k, v, np.full(6, -1), [0, 6], pk, pv, [0, 7], 0.3)
    want = osh.attn(q, k, v, np.arange(7), pk, pv, [0, 7], [0, 6], 0.3)
    assert all(np.allclose(a, b, atol=1e-12) for a, b in zip(got, want))


def test_siblings_do_not_see_each_other():
    q, k, v, pk, pv = make(3, 5, 3)
    parent = np.array([-1, 0, 0, 1, 2])
    assert otr.path(parent, 4) == [0, 2, 4] and otr.path(parent, 3) == [0, 1, 3] and otr.path([-1, 5, -9], 1) == [1]
    a = otr.attn(q, k, v, parent, [0, 5], pk, pv, [0, 3], 0.5)[0]
    k2, v2 = k.copy(), v.copy()
    k2[1], v2[1] = 9, 9                      # node 1: seen by itself and node 3 only
    b = otr.attn(q, k2, v2, parent, [0, 5], pk, pv, [0, 3], 0.5)[0]
    assert [bool(np.allclose(a[i], b[i])) for i in range(5)] == [True, False, True, False, True]
