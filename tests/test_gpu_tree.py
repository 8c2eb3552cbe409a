"""GPU parity of bg_tree_attn (through the C ABI) with the fp64 oracle, and its edges: chains, stars, deep and wide
trees, requests without prefix or nodes, cut key ranges, bad parents and offsets, planned runs, streams and graphs."""
import math

import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from attention_packed_varlen_causal_gb300 import workloads as wl
from oracle import tree as otr
from tests.helpers import from_dev, i32_dev, to_dev
from tests.test_gpu_shared import SENTINEL, assert_close, f64, sentinel_out

pytestmark = pytest.mark.gpu

HEADS = [(16, 8, 128), (14, 2, 64), (3, 3, 64), (4, 1, 128), (32, 8, 128), (16, 1, 64)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


def grow(rng, n, kind):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] * n
    if kind == "comb":                     # two interleaved chains
        return [i - 2 if i > 1 else -1 for i in range(n)]
    return [int(rng.integers(-1 if rng.random() < 0.1 else max(-1, i - 9), i)) if i else -1 for i in range(n)]


def make(seed, prefix, nodes, Hq, Hkv, d, kind="random", q_scale=1.0):
    rng = np.random.default_rng(seed)

    def cu(x):
        return np.concatenate(([0], np.cumsum(x))).astype(np.int32)

    def normal(n, h, s=1.0):
        return wl.bf16_bits_from_f32(s * rng.standard_normal((n, h, d), dtype=np.float32))

    x = dict(cu=cu(nodes), cup=cu(prefix), Hq=Hq, Hkv=Hkv, d=d, max_nodes=max(nodes), max_prefix=max(prefix),
             scale=1 / math.sqrt(d), parent=np.array([p for n in nodes for p in grow(rng, n, kind)], np.int32))
    T, P = sum(nodes), sum(prefix)
    x.update(q=normal(T, Hq, q_scale), k=normal(T, Hkv), v=normal(T, Hkv), pk=normal(P, Hkv), pv=normal(P, Hkv))
    return x


def device(x):
    t = {n: to_dev(x[n]) for n in ("q", "k", "v", "pk", "pv")}
    t.update({n: i32_dev(x[n]) for n in ("cu", "cup", "parent")})
    return t


def workspace(x):
    import torch
    n = bg.bg_tree_attn_workspace_size(len(x["cu"]) - 1, int(x["cu"][-1]), x["max_nodes"], x["max_prefix"], x["Hq"],
                                       x["Hkv"], x["d"])
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def call(x, t, out, *, ws=None, planned=False, **kw):
    fn = bg.bg_tree_attn_planned if planned else bg.bg_tree_attn
    return fn(t["q"], t["k"], t["v"], t["parent"], t["cu"], x["max_nodes"], t["pk"], t["pv"], t["cup"], x["max_prefix"], out,
              scale=x["scale"], workspace=workspace(x) if ws is None else ws, **kw)


def plan(x, t, ws, **kw):
    bg.bg_tree_plan(t["parent"], t["cu"], x["max_nodes"], t["cup"], int(x["cup"][-1]), x["max_prefix"], x["Hq"], x["Hkv"],
                    x["d"], workspace=ws, **kw)


def reference(x, softcap=0.0):
    return otr.attn(f64(x["q"]), f64(x["k"]), f64(x["v"]), x["parent"], x["cu"], f64(x["pk"]), f64(x["pv"]), x["cup"],
                    x["scale"], softcap=softcap)


def check(x, softcap=0.0, what=""):
    import torch
    rows = int(x["cu"][-1])
    full, out = sentinel_out((rows, x["Hq"], x["d"]))
    lse = torch.full((rows, x["Hq"]), 77.0, dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(x, device(x), out, lse=lse, softcap=softcap, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0, what
    assert (full.cpu().numpy()[rows * x["Hq"] * x["d"]:] == SENTINEL).all(), what
    assert_close(from_dev(out), lse.cpu().numpy().astype(np.float64), reference(x, softcap), what, softcap)


PACKINGS = {
    "one": ([100], [1]),
    "small": ([300, 0, 129, 5], [13, 7, 64, 1]),
    "tiles": ([128, 1, 256, 0], [127, 128, 129, 130]),
    "empty": ([50, 0, 0, 77], [0, 3, 0, 9]),
    "cuts": ([3000, 1500], [26, 40]),
    "wide": ([200], [300]),
}


@pytest.mark.parametrize("softcap", [0.0, 30.0, 100.0])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "h%d_%d_d%d" % h)
@pytest.mark.parametrize("packing", PACKINGS)
def test_parity(packing, heads, softcap):
    check(make(1, *PACKINGS[packing], *heads, q_scale=4.0 if softcap else 1.0), softcap, f"{packing} {heads}")


@pytest.mark.parametrize("kind", ["chain", "star", "comb"])
@pytest.mark.parametrize("heads", HEADS[:2], ids=lambda h: "h%d_%d_d%d" % h)
def test_shapes_of_trees(heads, kind):
    check(make(2, [200, 0], [150, 31], *heads, kind=kind), what=kind)


@pytest.mark.parametrize("kind", ["chain", "random", "star"])
def test_largest_trees(kind):
    check(make(3, [40, 0], [bg.BG_MAX_TREE, bg.BG_MAX_TREE - 1], 2, 2, 64, kind=kind), what=kind)


def test_every_number_of_nodes():
    check(make(4, [5 * (i % 7) for i in range(70)], list(range(1, 71)), 4, 2, 64))


def test_long_prefix():
    check(make(5, [20000, 9000], [64, 33], 16, 8, 128))


def test_many_requests():
    """More requests than the plan holds in shared memory, and more work items than CTAs."""
    check(make(6, [(i * 37) % 50 for i in range(700)], [1 + i % 5 for i in range(700)], 2, 1, 64))


def test_many_nodes_of_a_few_rows():
    check(make(7, [3] * 4200, [1] * 4200, 2, 2, 64))


def test_chain_is_shared_prefill():
    """Bit for bit what bg_shared_prefill_attn gives for one sample per request."""
    import torch
    x = make(8, [300, 1000, 0], [40, 130, 77], 16, 8, 128, kind="chain")
    t = device(x)
    a, b = torch.empty_like(t["q"]), torch.empty_like(t["q"])
    call(x, t, a)
    ws = torch.empty(bg.bg_shared_attn_workspace_size(3, 3, 247, 130, 1000, 16, 8, 128), dtype=torch.uint8, device="cuda")
    bg.bg_shared_prefill_attn(t["q"], t["k"], t["v"], t["cu"], 130, t["pk"], t["pv"], t["cup"], 1000, i32_dev(np.arange(4)), b,
                              scale=x["scale"], workspace=ws)
    assert torch.equal(a, b)


@pytest.mark.parametrize("n", [200, 3000], ids=["whole", "split"])
def test_nodes_without_prefix_tiles_of_minus_infinity(n):
    """Keys of the prefix and of some ancestors whose scores are -inf have weight 0."""
    x = make(9, [n], [40], 14, 2, 64)
    x["q"][:, :, 0] = 0x3F80
    x["pk"][:n - 10, :, 0] = 0xFF80
    x["k"][5:20, :, 0] = 0xFF80
    import torch
    out = torch.zeros((40, 14, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((40, 14), device="cuda")
    call(x, device(x), out, lse=lse)
    y = {m: f64(x[m]) for m in ("q", "k", "v", "pk", "pv")}
    with np.errstate(invalid="ignore"):
        o, l, A, B = otr.attn(y["q"], y["k"], y["v"], x["parent"], x["cu"], y["pk"], y["pv"], x["cup"], x["scale"])
    B[~np.isfinite(B)] = np.nanmax(np.where(np.isfinite(B), B, 0)) + 20
    assert_close(from_dev(out), lse.cpu().numpy().astype(np.float64), (o, l, A, B), "hidden keys")


def test_bad_parents_count_as_roots():
    import torch
    x = make(10, [70, 3], [50, 20], 16, 8, 128)
    bad = x["parent"].copy()
    bad[7], bad[20], bad[50], bad[60] = 7, 30, -2, 2147483647       # itself, a later one, and out of range
    x["parent"] = bad
    t = device(x)
    out, st = torch.empty_like(t["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    call(x, t, out, dev_status=st)
    assert int(st.item()) == bg.BG_DEVSTAT_PARENT
    assert_close(from_dev(out), None, reference(x), "bad parents")
    call(x, t, out)


@pytest.mark.parametrize("name,bad,bit", [
    ("cu", [0, 5, 4, 30], "BG_DEVSTAT_CU_SEQLENS"), ("cu", [1, 5, 9, 30], "BG_DEVSTAT_CU_SEQLENS"),
    ("cu", [0, 5, 9, 31], "BG_DEVSTAT_CU_SEQLENS"), ("cu", [0, -3, 9, 30], "BG_DEVSTAT_CU_SEQLENS"),
    ("cu", [0, 5, 9, 29], "BG_DEVSTAT_CU_SEQLENS"), ("cu", [0, 0, 0, 30], "BG_DEVSTAT_SEQ_TOO_LONG"),
    ("cup", [0, 9, 8, 60], "BG_DEVSTAT_CU_PROMPT"), ("cup", [0, 50, 55, 61], "BG_DEVSTAT_CU_PROMPT")], ids=str)
def test_bad_offsets(name, bad, bit):
    import torch
    x = make(11, [20, 20, 20], [10, 12, 8], 4, 2, 64)
    t = device(x)
    t[name] = i32_dev(np.array(bad))
    full, out = sentinel_out((30, 4, 64))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = workspace(x)
    call(x, t, out, ws=ws, dev_status=st)
    assert int(st.item()) & getattr(bg, bit)
    plan(x, t, ws)
    call(x, t, out, ws=ws, planned=True)
    torch.cuda.synchronize()
    assert (full == SENTINEL).all()


def test_non_finite_rows_stay_in_their_request():
    import torch
    x = make(12, [145, 150, 177], [20, 33, 70], 16, 8, 128)
    outs = []
    for poison in (False, True):
        t = device(x)
        if poison:
            for n, c in (("k", x["cu"]), ("v", x["cu"]), ("pk", x["cup"]), ("pv", x["cup"])):
                t[n][c[1]:c[2]] = float("nan") if n != "v" else float("inf")
        out = torch.zeros_like(t["q"])
        call(x, t, out)
        outs.append(out)
    c = x["cu"]
    assert torch.equal(outs[0][:c[1]], outs[1][:c[1]]) and torch.equal(outs[0][c[2]:], outs[1][c[2]:])


def test_non_finite_keys_reach_descendants_only():
    """Scores of nodes that a node does not descend from are masked, NaN and infinite ones too."""
    import torch
    for heads, softcap in ((HEADS[0], 0.0), (HEADS[1], 30.0), (HEADS[1], 100.0), (HEADS[1], 0.0)):
        x = make(13, [60], [140], *heads, kind="comb")
        t = device(x)
        clean, out = torch.zeros_like(t["q"]), torch.zeros_like(t["q"])
        call(x, t, clean, softcap=softcap)
        t["k"][1::2] = float("nan")
        t["k"][3::4] = float("inf")
        call(x, t, out, softcap=softcap)
        assert torch.equal(out[0::2], clean[0::2])


def test_planned_runs():
    """One plan, several layers; sizes that differ and other calls' plans are refused."""
    import torch
    xs = [make(14, [900, 40], [33, 12], 16, 8, 128) for _ in range(1)] + [make(15, [900, 40], [33, 12], 16, 8, 128)]
    xs[1]["parent"] = xs[0]["parent"]
    ts = [device(x) for x in xs]
    ws = workspace(xs[0])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan(xs[0], ts[0], ws, dev_status=st)
    for x, t in zip(xs, ts):
        one, two = torch.empty_like(t["q"]), torch.empty_like(t["q"])
        call(x, t, two, ws=ws, planned=True, dev_status=st)
        call(x, t, one)
        assert torch.equal(one, two)
    assert int(st.item()) == 0
    x, t = xs[0], ts[0]
    full, out = sentinel_out(t["q"].shape)
    call(dict(x, max_prefix=901), t, out, ws=workspace(dict(x, max_prefix=901)).copy_(
        torch.cat((ws, ws))[:workspace(dict(x, max_prefix=901)).numel()]), planned=True, dev_status=st)
    assert int(st.item()) == bg.BG_DEVSTAT_PLAN and (full == SENTINEL).all()
    # the plan of a shared prefill of the same sizes is another one
    st.zero_()
    cug = i32_dev(np.arange(3))
    big = torch.empty(max(ws.numel(), bg.bg_shared_attn_workspace_size(2, 2, 45, 33, 900, 16, 8, 128)), dtype=torch.uint8,
                      device="cuda")
    bg.bg_shared_prefill_plan(t["cu"], 45, 33, t["cup"], 940, 900, cug, 16, 8, 128, workspace=big)
    call(x, t, out, ws=big, planned=True, dev_status=st)
    assert int(st.item()) == bg.BG_DEVSTAT_PLAN and (full == SENTINEL).all()
    st.zero_()
    plan(x, t, big)
    bg.bg_shared_prefill_attn_planned(t["q"], t["k"], t["v"], t["cu"], 33, t["pk"], t["pv"], t["cup"], 900, cug, out,
                                      workspace=big, dev_status=st)
    assert int(st.item()) == bg.BG_DEVSTAT_PLAN and (full == SENTINEL).all()


def test_streams_and_graphs_that_share_a_workspace():
    import torch
    xs = [make(16, [3000, 100], [30, 61], 16, 8, 128), make(17, [700], [90], 14, 2, 64)]
    ts = [device(x) for x in xs]
    want = [torch.empty_like(t["q"]) for t in ts]
    for x, t, w in zip(xs, ts, want):
        call(x, t, w)
    outs = [torch.zeros_like(t["q"]) for t in ts]
    wss = [workspace(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, t, o, ws, s in zip(xs, ts, outs, wss, streams):
            call(x, t, o, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    ws = max(wss, key=lambda w: w.numel())
    graphs = []
    for x, t, o in zip(xs, ts, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(x, t, o, ws=ws)
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # a replay on another tree
    ts[0]["parent"].copy_(i32_dev(np.array([i - 1 for i in range(30)] + [-1] * 61)))
    graphs[0].replay()
    call(xs[0], ts[0], want[0])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0])


@pytest.mark.parametrize("heads", HEADS[:2], ids=lambda h: "h%d_%d_d%d" % h)
def test_without_any_prefix(heads):
    """prefix_k and prefix_v are None: nodes see their paths alone."""
    import torch
    x = make(18, [0, 0, 0], [40, 1, 200], *heads)
    t = device(x)
    out = torch.empty_like(t["q"])
    bg.bg_tree_attn(t["q"], t["k"], t["v"], t["parent"], t["cu"], 200, None, None, t["cup"], 0, out, scale=x["scale"],
                    workspace=workspace(x))
    assert_close(from_dev(out), None, reference(x), "no prefix")
    roots = x["parent"] == -1
    same = out[torch.from_numpy(np.flatnonzero(roots)).cuda()]
    v = t["v"][torch.from_numpy(np.flatnonzero(roots)).cuda()].repeat_interleave(heads[0] // heads[1], 1)
    assert torch.equal(same, v)                       # a root's only key is its own


def test_no_nodes():
    import torch
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    z = i32_dev(np.zeros(3))
    ws = torch.empty(max(256, bg.bg_tree_attn_workspace_size(2, 0, 0, 10, 4, 2, 64)), dtype=torch.uint8, device="cuda")
    bg.bg_tree_attn(e, k, k, i32_dev(np.zeros(0)), z, 0, None, None, z, 10, e, workspace=ws)


@pytest.mark.parametrize("heads", [(128, 1, 64), (40, 20, 128), (7, 1, 128)], ids=lambda h: "h%d_%d_d%d" % h)
def test_other_head_counts(heads):
    for softcap in (0.0, 30.0):
        check(make(19, [140, 0, 1100], [9, 33, 5], *heads), softcap, f"heads {heads}")


def test_bounds_above_the_lengths():
    """max_nodes and max_prefix_len are upper bounds: the same bits as with the lengths themselves."""
    import torch
    x = make(20, [900, 33], [45, 12], 16, 8, 128)
    t = device(x)
    want, out = torch.empty_like(t["q"]), torch.empty_like(t["q"])
    call(x, t, want)
    assert_close(from_dev(want), None, reference(x), "exact bounds")
    y = dict(x, max_nodes=bg.BG_MAX_TREE)
    call(y, t, out)
    assert torch.equal(out, want)
    y["max_prefix"] = 4000
    call(y, t, out)
    assert_close(from_dev(out), None, reference(x), "loose bounds")
