"""Edges of the shared-prefix attention calls on the GPU: scores of -inf in part of a key range, weights that
one key dominates or at the ends of their range, queries without keys in planned runs, void plans, and a
model with capped scores."""
import math

import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from attention_packed_varlen_causal_gb300 import workloads as wl
from oracle import shared as sh
from tests.helpers import from_dev, i32_dev, to_dev
from tests.test_gpu_shared import assert_close, call, device, f64, make, reference, workspace

pytestmark = pytest.mark.gpu

HEADS = [(16, 8, 128), (14, 2, 64)]
ONE, NEG_INF = 0x3F80, 0xFF80            # bf16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


def run(x, last, softcap=0.0, **kw):
    """(out, lse) as fp64, and the device status."""
    import torch
    rows = len(x["cu"]) - 1 if last else int(x["cu"][-1])
    out = torch.zeros((rows, x["Hq"], x["d"]), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((rows, x["Hq"]), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(x, device(x), last, out, lse=lse, softcap=softcap, dev_status=st, **kw)
    torch.cuda.synchronize()
    return from_dev(out), lse.cpu().numpy().astype(np.float64), int(st.item())


def hide_prefix(x, n):
    """The first n prefix rows get scores of -inf: -inf in one place of K, 1 in that place of q."""
    x["q"][:, :, 0] = x["ql"][:, :, 0] = ONE
    x["pk"][:n, :, 0] = NEG_INF


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "h%d_%d_d%d" % h)
@pytest.mark.parametrize("where", ["front", "back"])
@pytest.mark.parametrize("n,hidden", [(4000, 2700), (600, 300)], ids=["split", "whole"])
def test_tiles_whose_scores_are_all_minus_infinity(n, hidden, where, heads, last):
    """Their weights are 0: the rest of the keys decides, as if these were not there."""
    x = make(41, [n], [[3, 1, 40]], *heads)
    assert (workspace(x).numel() > 1 << 20) == (n > 1000)    # room for partial results: the range is cut
    hide_prefix(x, hidden)
    y = dict(x, pk=np.ascontiguousarray(x["pk"][hidden:]), pv=np.ascontiguousarray(x["pv"][hidden:]),
             cup=np.array([0, n - hidden], np.int32))
    if where == "back":
        x["pk"], x["pv"] = (np.ascontiguousarray(np.concatenate((x[m][hidden:], x[m][:hidden]))) for m in ("pk", "pv"))
    out, lse, st = run(x, last)
    assert st == 0
    assert_close(out, lse, reference(y, last), f"{where} {heads} last={last}")


@pytest.mark.parametrize("n", [100, 4000], ids=["whole", "split"])
def test_queries_whose_scores_are_all_minus_infinity(n):
    """A softmax over nothing but -inf: NaN with a log-sum of -inf, whether the range is cut or not."""
    x = make(42, [n], [[0, 0]], 16, 8, 128)
    hide_prefix(x, n)
    out, lse, st = run(x, True)
    assert np.isnan(out).all() and (lse == -math.inf).all() and st == 0


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
@pytest.mark.parametrize("softcap", [0.0, 7.0, 30.0, 55.0, 56.0, 300.0])
def test_queries_of_one_key_return_its_value(softcap, last):
    """One key (the first token of a sample without a prefix): its weight cancels out, whatever rounding it
    had, and out is v bit for bit (what fp32 leaves is 2^-22 of it, far below half a bf16 step)."""
    x = make(43, [0, 0], [[1] * 30, [1, 5, 1]], 14, 2, 64, q_scale=8.0)
    out = run(x, last, softcap)[0]
    v = from_dev(device(x)["v"])
    rows = np.flatnonzero(np.diff(x["cu"]) == 1)
    at = x["cu"][rows]
    assert np.array_equal(out[rows if last else at], np.repeat(v[at], 7, axis=1))


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
@pytest.mark.parametrize("prefix", [700, 5000], ids=["whole", "split"])
def test_capped_queries_with_a_dominant_key(prefix, last):
    """A prefix key along the query has a score of about +50 (a weight of 1.098 2^72, half a bf16 step off), the
    others -50: the result is that key's v bit for bit (the others' weights add up to less than 2^-130 of it)."""
    d, Hq = 64, 4
    x = make(44, [prefix], [[2, 9]], Hq, 2, d)
    s = np.sign(np.random.default_rng(44).standard_normal(d)).astype(np.float32)
    big = wl.bf16_bits_from_f32(np.tile(16 * s, (1, 1, 1)))
    for n in ("q", "ql"):
        x[n][:] = big
    x["k"][:] = x["pk"][:] = wl.bf16_bits_from_f32(np.tile(-16 * s, (1, 1, 1)))
    x["pk"][prefix - 333] = big[0]
    out = run(x, last, 50.0)[0]
    v = from_dev(device(x)["pv"])[prefix - 333]
    assert np.array_equal(out, np.broadcast_to(np.repeat(v, 2, axis=0), out.shape))


@pytest.mark.parametrize("prefix,groups,max_prefix", [
    ([0, 40], [[0, 0], [3]], 40), ([0, 3000], [[0], [3, 1]], 3000), ([0, 0], [[0, 0], [0]], 0), ([0, 0], [[0], [0]], 9000)],
    ids=["dealt", "cut", "no_key_at_all", "no_key_and_a_large_bound"])
def test_planned_runs_report_queries_without_keys(prefix, groups, max_prefix):
    """Every run raises BG_DEVSTAT_EMPTY_ROW, not only the plan, and leaves those rows as they are."""
    import torch
    x = dict(make(45, prefix, groups, 16, 8, 128), max_prefix=max_prefix)
    t, ws = device(x), workspace(x)
    st = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(3)]
    bg.bg_shared_last_token_plan(t["cu"], int(x["cu"][-1]), x["max_seqlen"], t["cup"], int(x["cup"][-1]), max_prefix,
                                 t["cug"], 16, 8, 128, workspace=ws, dev_status=st[0])
    none = np.diff(x["cu"]) + np.repeat(np.diff(x["cup"]), np.diff(x["cug"])) == 0
    for i in (1, 2):
        out = torch.full((len(none), 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        call(x, t, True, out, ws=ws, planned=True, dev_status=st[i])
        got = from_dev(out)
        assert (got[none] == 7.0).all() and not (got[~none] == 7.0).all(axis=(1, 2)).any()
    assert [int(s.item()) for s in st] == [bg.BG_DEVSTAT_EMPTY_ROW] * 3


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
def test_void_plans_write_nothing(last):
    """A plan that a run has voided (the status word, the workspace's first) leaves every row of later runs,
    those of cut key ranges among them, until it is made anew."""
    import torch
    x = make(46, [3000, 20], [[3, 50], [30, 7]], 14, 2, 64)
    t, ws = device(x), workspace(x)
    plan = bg.bg_shared_last_token_plan if last else bg.bg_shared_prefill_plan
    args = (t["cu"], int(x["cu"][-1]), x["max_seqlen"], t["cup"], int(x["cup"][-1]), x["max_prefix"], t["cug"], 14, 2, 64)
    outs = [torch.zeros_like(t["ql"] if last else t["q"]) for _ in range(3)]
    plan(*args, workspace=ws)
    call(x, t, last, outs[0], ws=ws, planned=True)
    ws[:4].view(torch.int32).fill_(bg.BG_DEVSTAT_TIMEOUT)
    call(x, t, last, outs[1], ws=ws, planned=True)
    plan(*args, workspace=ws)
    call(x, t, last, outs[2], ws=ws, planned=True)
    assert outs[0].any() and not outs[1].any() and torch.equal(outs[2], outs[0])


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
@pytest.mark.parametrize("sign,v_lo", [(1, 2.0 ** 29), (-1, 2.0 ** -46)], ids=["at_cap", "at_minus_cap"])
def test_ends_of_the_range_of_v_under_a_fixed_reference(sign, v_lo, last):
    """Cap 55, every score at one end: weights of 2^79.3 with |v| next to 2^30, of 2^-79.3 with |v| from 2^-46."""
    x = make(47, [300], [[5, 40]], 4, 2, 64)
    rng = np.random.default_rng(47)
    s = np.sign(rng.standard_normal(64)).astype(np.float32)
    for n in ("q", "ql"):
        x[n][:] = wl.bf16_bits_from_f32(np.tile(16 * s, (1, 1, 1)))
    for n in ("k", "pk"):
        x[n][:] = wl.bf16_bits_from_f32(np.tile(sign * 16 * s, (1, 1, 1)))
    for n in ("v", "pv"):
        v = v_lo * rng.uniform(1, 1.99, x[n].shape) * np.sign(rng.standard_normal(x[n].shape))
        x[n] = wl.bf16_bits_from_f32(v.astype(np.float32))
    out, lse, _ = run(x, last, 55.0)
    assert_close(out, lse, reference(x, last, 55.0), "ends of the range", 55.0)


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "h%d_%d_d%d" % h)
def test_capped_model_from_prefix_to_samples(heads):
    """A model with capped scores: the prefixes' rows as samples of requests without a prefix, then the samples
    over the same K and V, against whole sequences [prefix ; sample] of capped scores."""
    import torch
    prefix, groups, cap = [150, 1, 33], [[20, 1, 64], [7, 130], [3, 3]], 30.0
    Hq, Hkv, d = heads
    x = make(48, prefix, groups, *heads, q_scale=8.0)
    t = device(x)
    pq = wl.bf16_bits_from_f32(8 * np.random.default_rng(49).standard_normal((184, Hq, d), dtype=np.float32))
    pout, out = (torch.zeros((n, Hq, d), dtype=torch.bfloat16, device="cuda") for n in (184, int(x["cu"][-1])))
    none, each = i32_dev(np.zeros(4, np.int32)), i32_dev(np.arange(4, dtype=np.int32))
    ws = torch.empty(bg.bg_shared_attn_workspace_size(3, 3, 184, 150, 0, *heads), dtype=torch.uint8, device="cuda")
    bg.bg_shared_prefill_attn(to_dev(pq), t["pk"], t["pv"], t["cup"], 150, None, None, none, 0, each, pout,
                              scale=x["scale"], softcap=cap, workspace=ws)
    call(x, t, False, out, softcap=cap)
    # whole sequences: every prefix in front of each of its samples
    seqs, at = [], 0
    for r, group in enumerate(groups):
        for n in group:
            seqs.append((slice(x["cup"][r], x["cup"][r + 1]), slice(at, at + n)))
            at += n
    whole = {n: np.concatenate([np.concatenate((f64(a)[p], f64(b)[s])) for p, s in seqs])
             for n, a, b in (("q", pq, x["q"]), ("k", x["pk"], x["k"]), ("v", x["pv"], x["v"]))}
    lens = [p.stop - p.start + s.stop - s.start for p, s in seqs]
    cu = np.concatenate(([0], np.cumsum(lens)))
    empty = whole["k"][:0]
    ref = sh.attn(whole["q"], whole["k"], whole["v"], cu, empty, empty, np.zeros(2, int), np.array([0, len(seqs)]),
                  x["scale"], softcap=cap)
    both = np.concatenate([np.concatenate((from_dev(pout)[p], from_dev(out)[s])) for p, s in seqs])
    assert_close(both, None, ref, "capped model", cap)
