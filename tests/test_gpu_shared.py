"""GPU parity of bg_shared_prefill_attn and bg_shared_last_token_attn (through the C ABI) with the
fp64 oracle on the same bf16 inputs, and their behaviour at the edges: requests without prefix or
samples, samples without rows, queries without keys, split key ranges, non-finite neighbours, bad
offsets, planned runs, streams and graphs."""
import math

import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from attention_packed_varlen_causal_gb300 import workloads as wl
from oracle import shared as sh
from tests.helpers import from_dev, i32_dev, to_dev

pytestmark = pytest.mark.gpu

SENTINEL = 0x7FC1                 # a bf16 NaN pattern that the kernels never write
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


def make(seed, prefix, groups, Hq, Hkv, d, q_scale=1.0):
    rng = np.random.default_rng(seed)
    lens = [n for g in groups for n in g]

    def cu(x):
        return np.concatenate(([0], np.cumsum(x))).astype(np.int32)

    x = dict(cu=cu(lens), cup=cu(prefix), cug=cu([len(g) for g in groups]), Hq=Hq, Hkv=Hkv, d=d,
             max_seqlen=max(lens, default=0), max_prefix=max(prefix, default=0), scale=1 / math.sqrt(d))
    T, P = int(x["cu"][-1]), int(x["cup"][-1])

    def normal(n, h, s=1.0):
        return wl.bf16_bits_from_f32(s * rng.standard_normal((n, h, d), dtype=np.float32))

    x.update(q=normal(T, Hq, q_scale), ql=normal(len(lens), Hq, q_scale), k=normal(T, Hkv), v=normal(T, Hkv),
             pk=normal(P, Hkv), pv=normal(P, Hkv))
    return x


def f64(bits):
    return wl.bf16_bits_to_f32(bits).astype(np.float64)


def device(x):
    t = {n: to_dev(x[n]) for n in ("q", "ql", "k", "v", "pk", "pv")}
    t.update({n: i32_dev(x[n]) for n in ("cu", "cup", "cug")})
    return t


def workspace(x):
    import torch
    n = bg.bg_shared_attn_workspace_size(len(x["cug"]) - 1, len(x["cu"]) - 1, int(x["cu"][-1]), x["max_seqlen"],
                                         x["max_prefix"], x["Hq"], x["Hkv"], x["d"])
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def sentinel_out(shape):
    import torch
    n = int(np.prod(shape))
    full = torch.full((n + GUARD,), SENTINEL, dtype=torch.int16, device="cuda")
    return full, full[:n].view(torch.bfloat16).view(*shape)


def call(x, t, last, out, *, lse=None, softcap=0.0, ws=None, planned=False, **kw):
    name = ("bg_shared_last_token_attn" if last else "bg_shared_prefill_attn") + ("_planned" if planned else "")
    return getattr(bg, name)(t["ql"] if last else t["q"], t["k"], t["v"], t["cu"], x["max_seqlen"], t["pk"], t["pv"],
                             t["cup"], x["max_prefix"], t["cug"], out, lse=lse, scale=x["scale"], softcap=softcap,
                             workspace=workspace(x) if ws is None else ws, **kw)


def reference(x, last, softcap=0.0):
    return sh.attn(f64(x["ql"] if last else x["q"]), f64(x["k"]), f64(x["v"]), x["cu"], f64(x["pk"]), f64(x["pv"]),
                   x["cup"], x["cug"], x["scale"], softcap=softcap, last=last)


def assert_close(got, lse, ref, what, softcap=0.0):
    """Element-wise bounds from the kernel's arithmetic.  With A the weighted mean of |v| and o the
    exact value: every weight is rounded to bf16 once (half a step, 2^-8 of it: A 2^-8 in the sum),
    the sum it is divided by carries the rounding of the tiles' largest weights (|o| 2^-8), and the
    result is rounded to bf16 (|o| 2^-8).  A score is a sum of d fp32 products: its error is below
    2^-23 d B with B = scale * sum |q_i k_i|, and moves a weight, the sum and lse by that much (twice
    over: numerator and sum); 2^-18 covers the exponential and the fp32 sums.  A capped score is the
    difference of two numbers of the cap's size from an exponential (2^-22), a sum, a product of four
    and a reciprocal: an error of 2^-20 of the cap; above 55 small scores come from the series of tanh
    (four multiply-adds, 2^-21 of the score), the others are at least 0.29 of the cap, so that the
    error is below 2^-18 of the score, which B bounds."""
    o, l64, A, B = ref
    live = np.isfinite(l64)
    d = o.shape[-1]
    s_err = (2.0 ** -23 * d * B + 2.0 ** -18 * (1 + (np.minimum(B, softcap) if softcap > 55 else softcap / 4)))[..., None]
    tol = 2.0 ** -8 * (A + 2 * np.abs(o)) * (1 + 2.0 ** -7) + 2 * s_err * A
    err = np.abs(got - o)
    assert np.isfinite(got[live]).all(), what
    worst = (err - tol)[live].max() if live.any() else -1.0
    assert worst <= 0, f"{what}: error above its bound by {worst:.3e}"
    if lse is not None:
        lt = s_err[..., 0] + 2.0 ** -22 * np.abs(np.where(live, l64, 0))
        assert (np.abs(lse - l64)[live] <= lt[live]).all(), f"{what}: lse {np.abs(lse - l64)[live].max():.3e}"


def check(x, last, softcap=0.0, what=""):
    import torch
    rows = len(x["cu"]) - 1 if last else int(x["cu"][-1])
    full, out = sentinel_out((rows, x["Hq"], x["d"]))
    lse = torch.full((rows, x["Hq"]), 77.0, dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(x, device(x), last, out, lse=lse, softcap=softcap, dev_status=st)
    torch.cuda.synchronize()
    ref = reference(x, last, softcap)
    got, lse = from_dev(out), lse.cpu().numpy().astype(np.float64)
    bits = full.cpu().numpy()
    dead = ~np.isfinite(ref[1])
    assert (bits[rows * x["Hq"] * x["d"]:] == SENTINEL).all(), f"{what}: write past the end of out"
    assert (bits[:rows * x["Hq"] * x["d"]].reshape(rows, x["Hq"], x["d"])[dead] == SENTINEL).all() and \
        (lse[dead] == 77.0).all(), f"{what}: a query without keys was written"
    assert int(st.item()) == (bg.BG_DEVSTAT_EMPTY_ROW if dead.any() else 0)
    assert_close(got, lse, ref, what, softcap)


HEADS = [(16, 8, 128), (14, 2, 64), (4, 4, 64), (21, 3, 128), (8, 1, 128), (2, 2, 128), (40, 1, 64), (130, 2, 64),
         (128, 1, 64)]
# prefix lengths and sample lengths around the 16-, 64- and 128-key steps, empty ones among them
PACKINGS = {
    "one": ([1], [[1]]),
    "short": ([5, 0, 17], [[1, 2, 3], [7, 1], [16, 15, 17]]),
    "edges": ([127, 128, 129, 64], [[63, 1, 65], [128], [127, 2], [64, 64, 64]]),
    "empties": ([40, 0, 33, 0, 0], [[0, 3, 0, 0], [], [0], [0, 9], [5, 0, 0]]),
    "no_prefix": ([0, 0], [[130, 1, 40], [257]]),
    "many_samples": ([200], [[3, 1, 4, 1, 5, 9, 2, 6] * 9]),
    "long_sample": ([70, 300], [[400, 30], [1, 1, 1]]),
}


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "h%d_%d_d%d" % h)
@pytest.mark.parametrize("packing", PACKINGS)
def test_packings(packing, heads, last):
    prefix, groups = PACKINGS[packing]
    if last is False and sum(map(sum, groups)) == 0:
        pytest.skip("no tokens")
    Hq = heads[0]
    if Hq > 40 and packing in ("long_sample", "many_samples", "no_prefix", "edges"):
        groups = [g[:2] for g in groups]                     # keeps the fp64 reference short
    check(make(11, prefix, groups, *heads), last, what=f"{packing} {heads} last={last}")


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
@pytest.mark.parametrize("heads", [(16, 8, 128), (14, 2, 64), (4, 4, 64)], ids=lambda h: "h%d_%d_d%d" % h)
@pytest.mark.parametrize("softcap,q_scale", [(30.0, 8.0), (20.0, 1.0), (30.0, 60.0), (55.0, 60.0), (56.0, 8.0),
                                             (1000.0, 60.0), (1e6, 8.0), (0.01, 8.0)])
def test_capped(softcap, q_scale, heads, last):
    """Scores far below, around and far above the cap."""
    prefix, groups = PACKINGS["edges"]
    check(make(12, prefix, groups, *heads, q_scale=q_scale), last, softcap=softcap, what=f"cap {softcap} {q_scale}")


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
@pytest.mark.parametrize("heads", [(16, 8, 128), (14, 2, 64)], ids=lambda h: "h%d_%d_d%d" % h)
def test_split_key_ranges(heads, last):
    """Few queries over long prefixes: the key ranges are split and joined (with an empty prefix and
    a sample without rows among them, so that some pieces hold no key of some queries)."""
    x = make(13, [5000, 0, 1025], [[3, 0, 1], [1600, 0], [2, 40]], *heads)
    assert workspace(x).numel() > (1 << 20)                  # partial results are part of it
    check(x, last, what=f"split {heads}")
    check(make(14, [4096], [[1]], *heads, q_scale=4.0), last, softcap=30.0, what=f"split one {heads}")


def test_peaked_scores_and_growing_maximum():
    """Scores whose maximum grows by far more than 2^8 from tile to tile, and rows of one dominant key."""
    x = make(15, [500], [[120, 300]], 4, 2, 64, q_scale=30.0)
    ramp = np.linspace(0.05, 2.0, 500)[:, None, None]
    x["pk"] = wl.bf16_bits_from_f32((f64(x["pk"]) * ramp).astype(np.float32))
    for last in (False, True):
        check(x, last, what="ramp")


@pytest.mark.parametrize("softcap", [0.0, 30.0, 100.0])
@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
def test_non_finite_neighbours_stay_in_their_request(last, softcap):
    """K and V of the middle request are NaN and infinities; the others' outputs are bit for bit
    what they are without it."""
    import torch
    x = make(16, [45, 50, 77], [[20, 3], [9, 30], [70, 1]], 16, 8, 128)
    rows = len(x["cu"]) - 1 if last else int(x["cu"][-1])
    outs = []
    for bad in (False, True):
        t = device(x)
        if bad:
            for n, c in (("k", x["cu"][x["cug"]]), ("v", x["cu"][x["cug"]]), ("pk", x["cup"]), ("pv", x["cup"])):
                t[n][c[1]:c[2]] = float("nan") if n != "v" else float("inf")
        out = torch.zeros((rows, 16, 128), dtype=torch.bfloat16, device="cuda")
        call(x, t, last, out, softcap=softcap)
        outs.append(out)
    b = x["cug"] if last else x["cu"][x["cug"]]
    assert torch.equal(outs[0][:b[1]], outs[1][:b[1]]) and torch.equal(outs[0][b[2]:], outs[1][b[2]:])
    assert torch.isnan(outs[1][b[1]:b[2]].float()).all()


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
def test_planned_equals_one_call_and_is_deterministic(last):
    import torch
    x = make(17, [3000, 20], [[3, 50], [300, 7]], 14, 2, 64)
    t, ws = device(x), workspace(x)
    rows = len(x["cu"]) - 1 if last else int(x["cu"][-1])
    outs = [torch.zeros((rows, 14, 64), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    call(x, t, last, outs[0], ws=ws)
    call(x, t, last, outs[1])
    plan = bg.bg_shared_last_token_plan if last else bg.bg_shared_prefill_plan
    plan(t["cu"], int(x["cu"][-1]), x["max_seqlen"], t["cup"], int(x["cup"][-1]), x["max_prefix"], t["cug"], 14, 2, 64,
         workspace=ws)
    call(x, t, last, outs[2], ws=ws, planned=True)
    call(x, t, last, outs[3], ws=ws, planned=True)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    # a planned run of the other kind, or of another size, writes nothing and says so
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    other = torch.zeros((int(x["cu"][-1]) if last else len(x["cu"]) - 1, 14, 64), dtype=torch.bfloat16, device="cuda")
    call(x, t, not last, other, ws=ws, planned=True, dev_status=st)
    assert int(st.item()) == bg.BG_DEVSTAT_PLAN and not other.any()


def test_last_token_equals_the_prefill_rows():
    """The last row of every sample from both calls (both against the same queries)."""
    import torch
    x = make(18, [200, 31], [[5, 80, 1], [140, 3]], 16, 8, 128)
    ends = x["cu"][1:] - 1
    x["ql"] = np.ascontiguousarray(x["q"][ends])
    t = device(x)
    full = torch.zeros((int(x["cu"][-1]), 16, 128), dtype=torch.bfloat16, device="cuda")
    one = torch.zeros((len(ends), 16, 128), dtype=torch.bfloat16, device="cuda")
    call(x, t, False, full)
    call(x, t, True, one)
    ref = reference(x, True)
    assert_close(from_dev(one), None, ref, "last")
    assert_close(from_dev(full)[ends], None, ref, "prefill rows")


@pytest.mark.parametrize("which,bad,bit", [
    ("cu", lambda c: c[::-1].copy(), "CU_SEQLENS"), ("cu", lambda c: c + 1, "CU_SEQLENS"),
    ("cup", lambda c: c + 1, "CU_PROMPT"), ("cup", lambda c: np.minimum(c, 3), "CU_PROMPT"),
    ("cug", lambda c: c[::-1].copy(), "GROUP"), ("cug", lambda c: np.minimum(c, 2), "GROUP"),
    ("cug", lambda c: c - 2, "GROUP"), ("cug", lambda c: c * 1000, "GROUP")])
@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
def test_bad_offsets_write_nothing(which, bad, bit, last):
    import torch
    x = make(19, [10, 30], [[4, 6], [7, 8]], 4, 2, 64)
    t = device(x)
    t[which] = i32_dev(bad(x[which]))
    rows = 4 if last else 25
    full, out = sentinel_out((rows, 4, 64))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(x, t, last, out, dev_status=st)
    assert int(st.item()) & getattr(bg, "BG_DEVSTAT_" + bit)
    assert (full == SENTINEL).all()


def test_lengths_above_their_bounds_are_reported():
    import torch
    x = make(20, [10, 30], [[4, 6], [7, 8]], 4, 2, 64)
    for key, bit in (("max_seqlen", bg.BG_DEVSTAT_SEQ_TOO_LONG), ("max_prefix", bg.BG_DEVSTAT_CU_PROMPT)):
        y = dict(x)
        y[key] -= 1
        full, out = sentinel_out((25, 4, 64))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(y, device(x), False, out, dev_status=st)
        assert int(st.item()) == bit and (full == SENTINEL).all()


def test_no_prefix_tensor_and_out_on_a_16_byte_boundary():
    import torch
    x = make(21, [0, 0], [[30, 5], [61]], 6, 2, 64)
    t = device(x)
    buf = torch.zeros(96 * 6 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    out = buf[8:].view(96, 6, 64)
    assert out.data_ptr() % 32 == 16
    bg.bg_shared_prefill_attn(t["q"], t["k"], t["v"], t["cu"], x["max_seqlen"], None, None, t["cup"], 0, t["cug"], out,
                              scale=x["scale"], workspace=workspace(x))
    assert_close(from_dev(out), None, reference(x, False), "16-byte out")


def test_side_stream_and_graph_replay():
    """On a stream other than the default one, captured and replayed with new inputs in the same buffers."""
    import torch
    x, y = (make(s, [900, 2500], [[30, 5], [61, 200, 1]], 16, 8, 128) for s in (22, 23))
    t, ws = device(x), workspace(x)
    out = torch.zeros((297, 16, 128), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(x, t, False, out, ws=ws)
    side.synchronize()
    assert_close(from_dev(out), None, reference(x, False), "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(x, t, False, out, ws=ws)
        call(x, t, False, out, ws=ws)
    for z in (y, x):
        for n in ("q", "k", "v", "pk", "pv"):
            t[n].copy_(to_dev(z[n]))
        graph.replay()
        torch.cuda.synchronize()
        assert_close(from_dev(out), None, reference(z, False), "replay")


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
@pytest.mark.parametrize("num_groups,samples,heads", [(600, 2, (2, 2, 64)), (1300, 4, (4, 2, 64)), (3, 1500, (128, 1, 64))],
                         ids=["groups600", "groups1300_seqs5200", "entries_above_1024"])
def test_large_work_lists(num_groups, samples, heads, last):
    """More requests, samples and entries than the pre-pass holds in shared memory or handles at once."""
    rng = np.random.default_rng(24)
    groups = [rng.integers(0, 3, samples).tolist() for _ in range(num_groups)]
    prefix = rng.integers(0, 4, num_groups).tolist()
    check(make(24, prefix, groups, *heads), last, what=f"{num_groups} requests of {samples}")


def test_key_offsets_past_32_bits():
    """A prefix cache of more than 2^32 elements, of which the last request's rows count."""
    import torch
    x = make(25, [65000, 300], [[3, 40], [20]], 8, 8, 128)
    t = device(x)
    before = 65 * 65536                                     # rows of 65 requests without samples: 2^32 elements
    y = dict(x, cup=np.concatenate((np.arange(66) * 65536, before + x["cup"][1:])).astype(np.int32),
             cug=np.concatenate((np.zeros(65), x["cug"])).astype(np.int32), max_prefix=65536)
    P = int(y["cup"][-1])
    assert (P - 65300) * 8 * 128 > 1 << 32
    for n in ("pk", "pv"):
        big = torch.zeros((P, 8, 128), dtype=torch.bfloat16, device="cuda")
        big[before:] = t[n]
        t[n] = big
    t.update({n: i32_dev(y[n]) for n in ("cup", "cug")})
    for last in (False, True):
        out = torch.zeros((3 if last else 63, 8, 128), dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(y, t, last, out, dev_status=st)
        assert int(st.item()) == 0
        assert_close(from_dev(out), None, reference(x, last), "offsets past 32 bits")


@pytest.mark.parametrize("last", [False, True], ids=["prefill", "last"])
def test_query_offsets_past_31_bits(last):
    """Queries and outputs of more than 2^31 elements: samples of one token; the rows at both ends are compared."""
    import torch
    S, Hq, d, n = (1 << 18) + 77, 128, 64, 40
    x = make(26, [n], [[1] * 50], Hq, 1, d)
    t = device(x)
    gen = torch.Generator(device="cuda").manual_seed(26)
    q = torch.randn((S, Hq, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    assert q.numel() > 1 << 31
    k, v = (torch.randn((S, 1, d), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    cug = i32_dev(np.array([0, S], np.int32))
    out = torch.zeros_like(q)
    ws = torch.empty(bg.bg_shared_attn_workspace_size(1, S, S, 1, n, Hq, 1, d), dtype=torch.uint8, device="cuda")
    fn = bg.bg_shared_last_token_attn if last else bg.bg_shared_prefill_attn
    fn(q, k, v, cu, 1, t["pk"], t["pv"], t["cup"], n, cug, out, workspace=ws)
    for rows in (slice(0, 50), slice(S - 50, S)):
        y = {m: np.ascontiguousarray(a[rows].view(torch.int16).cpu().numpy().view(np.uint16))
             for m, a in (("q", q), ("k", k), ("v", v))}
        ref = sh.attn(f64(y["q"]), f64(y["k"]), f64(y["v"]), np.arange(51), f64(x["pk"]), f64(x["pv"]), x["cup"],
                      [0, 50], 1 / math.sqrt(d), last=last)
        assert_close(from_dev(out[rows].contiguous()), None, ref, f"rows {rows}")


def test_two_streams_and_shared_workspace_of_two_graphs():
    """Two problems at once on two streams, each with its workspace; then two captured graphs that
    share one workspace, replayed in turn on one stream."""
    import torch
    xs = [make(27, [3000, 100], [[30, 5], [61, 200, 1]], 16, 8, 128), make(28, [700], [[90, 1, 300]], 14, 2, 64)]
    ts = [device(x) for x in xs]
    outs = [[torch.zeros_like(t["ql"] if last else t["q"]) for last in (False, True)] for t in ts]
    sizes = [workspace(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, t, o, ws, st in zip(xs, ts, outs, sizes, streams):
            for last in (False, True):
                call(x, t, last, o[last], ws=ws, stream=st)
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        for last in (False, True):
            assert_close(from_dev(o[last]), None, reference(x, last), "two streams")
    ref = [[o.clone() for o in pair] for pair in outs]
    ws = max(sizes, key=lambda w: w.numel())
    graphs = []
    for x, t, o in zip(xs, ts, outs):
        for last in (False, True):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(x, t, last, o[last], ws=ws)
            graphs.append((g, o[last], ref[len(graphs) // 2][last]))
    for _ in range(2):
        for g, o, _ in graphs:
            o.zero_()
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for _, o, r in graphs)


PAIRED = {
    # most requests fill one query tile or less: two kv heads share an entry
    "batch": ([300, 0, 129, 255, 64, 300], [[30, 5, 60], [64, 1], [17] * 9, [90, 80, 1], [128], [0, 3]]),
    # entries of two tiles, of one (the rest of a request, its last rows), and of few rows
    "tiles": ([10, 7, 0], [[3, 9, 5] * 23, [4, 2] * 65, [6]]),
    # key ranges that several CTAs share
    "cuts": ([2000] * 5 + [0, 1999], [[3, 40, 1]] * 7),
}


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("heads", [(16, 8, 128), (14, 2, 64), (32, 16, 64), (48, 24, 128)], ids=lambda h: "h%d_%d_d%d" % h)
@pytest.mark.parametrize("packing", PAIRED)
def test_last_token_of_paired_heads(packing, heads, softcap):
    check(make(29, *PAIRED[packing], *heads), True, softcap=softcap, what=f"paired {packing} {heads}")


def test_paired_heads_keep_non_finite_rows_in_their_request():
    import torch
    x = make(30, [145, 150, 177], [[20, 3] * 8, [9, 30] * 8, [70, 1] * 4], 16, 8, 128)
    outs = []
    for bad in (False, True):
        t = device(x)
        if bad:
            for n, c in (("k", x["cu"][x["cug"]]), ("v", x["cu"][x["cug"]]), ("pk", x["cup"]), ("pv", x["cup"])):
                t[n][c[1]:c[2]] = float("nan") if n != "v" else float("inf")
        out = torch.zeros((len(x["cu"]) - 1, 16, 128), dtype=torch.bfloat16, device="cuda")
        call(x, t, True, out)
        outs.append(out)
    b = x["cug"]
    assert torch.equal(outs[0][:b[1]], outs[1][:b[1]]) and torch.equal(outs[0][b[2]:], outs[1][b[2]:])
    assert torch.isnan(outs[1][b[1]:b[2]].float()).all()


def test_last_token_of_samples_without_rows():
    """No sample has a row: every query sees its request's prefix only, and k and v are empty."""
    x = make(31, [40, 129, 0], [[0, 0, 0], [0], [0, 0]], 16, 8, 128)
    check(x, True, what="no own rows")
