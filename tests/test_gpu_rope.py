"""GPU parity of bg_packed_qk_norm_rope and bg_beam_qk_norm_rope (through the C ABI) with the fp64 oracle, and their
edges: strides, places in memory, far positions, several axes, partly rotated heads, values that are not finite."""
import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from oracle import rope as orp

pytestmark = pytest.mark.gpu

HEADS = [(16, 8, 128), (14, 2, 64), (3, 3, 128), (5, 1, 64), (1, 1, 128)]
SENTINEL = 0x7FC1                 # a bf16 NaN pattern that the kernels never write
GUARD = 1024


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


def frequencies(n, base=1e4):
    import torch
    return (base ** (-torch.arange(n, dtype=torch.float64) / n)).float().cuda()


def inputs(seed, rows, Hq, Hkv, d, *, axes=1, rot=None, norm=True, far=3000):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rot = d if rot is None else rot

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x = dict(Hq=Hq, Hkv=Hkv, d=d, qkv=normal(rows, (Hq + 2 * Hkv) * d).bfloat16(),
             positions=torch.randint(0, far, (axes, rows), generator=gen, device="cuda", dtype=torch.int32),
             kw=dict(inv_freq=frequencies(rot // 2)))
    if norm:
        x["kw"].update(q_weight=(1 + 0.3 * normal(d)).bfloat16(), k_weight=(1 + 0.3 * normal(d)).bfloat16())
    if axes > 1:
        x["kw"].update(axis_of=[i % axes for i in range(rot // 2)])
    return x


def split(x):
    q, k, v = x["qkv"].split((x["Hq"] * x["d"], x["Hkv"] * x["d"], x["Hkv"] * x["d"]), -1)
    return q.unflatten(-1, (x["Hq"], x["d"])), k.unflatten(-1, (x["Hkv"], x["d"])), v.unflatten(-1, (x["Hkv"], x["d"]))


def f64(t):
    return t.double().cpu().numpy()


def reference(x, t, weight, pos):
    kw = x["kw"]
    w = kw.get(weight)
    return orp.norm_rotate(f64(t), None if w is None else f64(w), kw.get("eps", 1e-6), kw.get("weight_offset", 0.0),
                           pos.cpu().numpy(), f64(kw["inv_freq"]), kw.get("axis_of"), kw.get("interleaved", False),
                           kw.get("rope_scale", 1.0))


def assert_close(got, ref, rope_scale=1.0, far=False):
    """An angle is off by at most 2^-17 (2^-15 where the position passes 2^24), cosine and sine by 2^-21 more, the
    norm's sum of d squares by 2^-24 d (half of it in the root), the products and sums by a few times 2^-24: together
    below 2^-16 (2^-14) of what the element is made of.  The result is rounded to bf16 once: half a step, 2^-8 of it."""
    out, size = ref
    e = (2.0 ** -14 if far else 2.0 ** -16) * size * max(1.0, abs(rope_scale))
    tol = e + 2.0 ** -8 * (np.abs(out) + e)
    err = np.abs(f64(got) - out)
    assert (err <= tol).all(), (err - tol).max()


def guarded(*shape):
    import torch
    n = int(np.prod(shape))
    full = torch.full((n + GUARD,), SENTINEL, dtype=torch.int16, device="cuda")
    return full, full[:n].view(torch.bfloat16).view(*shape)


def run(x, with_v=True):
    import torch
    q, k, v = split(x)
    outs = [guarded(*t.shape) for t in (q, k, v)]
    bg.bg_packed_qk_norm_rope(q, k, v if with_v else None, x["positions"], outs[0][1], outs[1][1],
                              outs[2][1] if with_v else None, **x["kw"])
    torch.cuda.synchronize()
    for (full, out), t in zip(outs, (q, k, v)):
        assert (full[t.numel():] == SENTINEL).all()
    return [o for _, o in outs]


def check(x, **kw):
    import torch
    q, k, v = split(x)
    out = run(x)
    scale = x["kw"].get("rope_scale", 1.0)
    assert_close(out[0], reference(x, q, "q_weight", x["positions"]), scale, **kw)
    assert_close(out[1], reference(x, k, "k_weight", x["positions"]), scale, **kw)
    assert torch.equal(out[2], v)
    return out


@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "h%d_%d_d%d" % h)
@pytest.mark.parametrize("rows", [1, 2, 37, 700])
def test_parity(rows, heads, interleaved, norm):
    x = inputs(1, rows, *heads, norm=norm)
    x["kw"]["interleaved"] = interleaved
    check(x)


def test_many_rows():
    """More rows than warps on the card, so that each warp takes several."""
    check(inputs(2, 20011, 14, 2, 64))


@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("heads", [(4, 2, 128), (7, 1, 64)], ids=lambda h: "h%d_%d_d%d" % h)
def test_a_large_batch_is_its_parts(heads, interleaved, norm):
    """Launches of many and of few tokens give the same bits."""
    import torch
    x = inputs(19, 26001, *heads, norm=norm, axes=2)
    x["kw"]["interleaved"] = interleaved
    whole = run(x)
    for a, b in ((0, 900), (12000, 12700), (25500, 26001)):
        part = run(dict(x, qkv=x["qkv"][a:b], positions=x["positions"][:, a:b].contiguous()))
        assert all(torch.equal(w[a:b], t) for w, t in zip(whole, part))


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("d,rot", [(128, 16), (128, 64), (128, 112), (64, 16), (64, 32), (64, 48)])
def test_partly_rotated(d, rot, interleaved):
    for norm in (False, True):
        x = inputs(3, 50, 6, 2, d, rot=rot, norm=norm)
        x["kw"]["interleaved"] = interleaved
        out = check(x)
        if not norm:                      # what does not turn is the input, bit for bit
            assert (out[0][..., rot:] == split(x)[0][..., rot:]).all()


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_several_axes(axes, d):
    for rot in (d, d // 2):
        check(inputs(4, 333, 8, 2, d, axes=axes, rot=rot))


def test_one_axis_as_a_vector_and_scaled():
    import torch
    x = inputs(5, 40, 4, 2, 128)
    x["kw"].update(rope_scale=1.25, eps=0.01, weight_offset=1.0)
    a = check(x)
    x["positions"] = x["positions"][0].contiguous()
    b = run(x)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
def test_far_positions(d):
    import torch
    x = inputs(6, 64, 4, 2, d)
    x["positions"][0, :16] = torch.tensor([0, 1, -1, 4095, 4096, 65535, 131071, -131072, 1 << 20, (1 << 20) + 1, 16777215,
                                           16777216, -16777216, 12345678, 8388609, -5], dtype=torch.int32)
    check(x)
    x["positions"][0, :8] = torch.tensor([2147483647, -2147483648, 16777217, 33554435, 1000000007, -1000000007, 1 << 30,
                                          (1 << 30) + 1], dtype=torch.int32)
    check(x, far=True)


def test_separate_strided_and_in_place():
    import torch
    x = inputs(7, 91, 16, 8, 128)
    want = run(x)
    q, k, v = (t.contiguous() for t in split(x))
    wide = torch.zeros((91, 8, 24, 128), dtype=torch.bfloat16, device="cuda")
    rows = wide[:, 3, 5:13]                         # every row of heads within a larger one
    rows.copy_(k)
    o = [torch.empty_like(t) for t in (q, k)]
    bg.bg_packed_qk_norm_rope(q, rows, None, x["positions"], *o, **x["kw"])
    assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    bg.bg_packed_qk_norm_rope(q, k, v, x["positions"], q, k, v, **x["kw"])
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), want))


def test_without_v():
    x = inputs(8, 33, 14, 2, 64)
    out = run(x, with_v=False)
    assert_close(out[0], reference(x, split(x)[0], "q_weight", x["positions"]))
    assert (out[2].view_as(out[2]).isnan()).all()


def test_non_finite_values_stay_in_their_head():
    import torch
    for norm in (False, True):
        x = inputs(9, 20, 4, 2, 64, rot=32, norm=norm)
        clean = run(x)
        q, k, v = split(x)
        q[3, 1, 2], q[7, 0, 60], k[5, 1, 0], v[2, 0, 0] = float("nan"), float("inf"), float("-inf"), float("nan")
        out = run(x)
        for t, places in ((0, [(3, 1), (7, 0)]), (1, [(5, 1)])):
            same = torch.ones(clean[t].shape[:2], dtype=torch.bool, device="cuda")
            for p in places:
                same[p] = False
            assert torch.equal(out[t][same], clean[t][same])
        if norm:
            assert out[0][3, 1].isnan().all()
        else:                             # an infinity that does not turn reaches no other element
            assert out[0][7, 0, 60] == float("inf") and out[0][7, 0, :60].isfinite().all()
        assert torch.equal(out[2].view(torch.int16), v.contiguous().view(torch.int16))


def test_zeros_and_large_values():
    """A head of zeros stays zeros; eps = 0 makes it NaN as the formula does; large values do not overflow the result."""
    import torch
    x = inputs(10, 12, 4, 2, 128)
    q, k, v = split(x)
    q[4] = 0
    k[:] *= 1e15
    out = check(x)
    assert (out[0][4] == 0).all()
    x["kw"]["eps"] = 0.0
    assert run(x)[0][4].isnan().all()


@pytest.mark.parametrize("R,W,slots,slot,step", [(1, 1, 1, 0, 0), (3, 100, 5, 2, 2), (2, 37, 16, 15, 40), (16, 400, 5, 4, 4)])
@pytest.mark.parametrize("heads", [(16, 8, 128), (14, 2, 64), (3, 3, 64)], ids=lambda h: "h%d_%d_d%d" % h)
def test_beams(heads, R, W, slots, slot, step):
    import torch
    Hq, Hkv, d = heads
    x = inputs(11, R * W, *heads)
    gen = torch.Generator(device="cuda").manual_seed(12)
    base = torch.randint(1, 500, (R,), generator=gen, device="cuda", dtype=torch.int32)
    q, k, v = (t.unflatten(0, (R, W)) for t in split(x))
    sk, sv = (torch.randn((R, W, slots, Hkv, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    before = sk.clone(), sv.clone()
    full, out = guarded(R, W, Hq, d)
    bg.bg_beam_qk_norm_rope(q, k, v, base, step, out, sk, sv, slot, **x["kw"])
    pos = (base + step).repeat_interleave(W)[None]
    assert_close(out.flatten(0, 1), reference(x, q.flatten(0, 1), "q_weight", pos))
    assert_close(sk[:, :, slot].flatten(0, 1), reference(x, k.flatten(0, 1), "k_weight", pos))
    assert torch.equal(sv[:, :, slot], v)
    others = [s for s in range(slots) if s != slot]
    assert torch.equal(sk[:, :, others], before[0][:, :, others]) and torch.equal(sv[:, :, others], before[1][:, :, others])
    assert (full[out.numel():] == SENTINEL).all()
    # the packed call at the same positions gives the same bits
    x["positions"] = pos
    p = run(x)
    assert torch.equal(p[0], out.flatten(0, 1)) and torch.equal(p[1], sk[:, :, slot].flatten(0, 1))


def test_beams_with_axes_and_in_place():
    """Three axes; then K and V that already lie in the slot."""
    import torch
    R, W, Hq, Hkv, d = 3, 10, 6, 2, 128
    x = inputs(13, R * W, Hq, Hkv, d, axes=3)
    base = torch.tensor([[5, 6, 7], [100, 0, 31], [9, 9, 2]], dtype=torch.int32, device="cuda")
    q, k, v = (t.unflatten(0, (R, W)) for t in split(x))
    sk, sv = (torch.zeros((R, W, 4, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.empty((R, W, Hq, d), dtype=torch.bfloat16, device="cuda")
    bg.bg_beam_qk_norm_rope(q, k, v, base, 3, out, sk, sv, 1, **x["kw"])
    pos = (base + 3).repeat_interleave(W, 1)
    assert_close(out.flatten(0, 1), reference(x, q.flatten(0, 1), "q_weight", pos))
    assert_close(sk[:, :, 1].flatten(0, 1), reference(x, k.flatten(0, 1), "k_weight", pos))
    ik, iv = torch.zeros_like(sk), torch.zeros_like(sv)
    ik[:, :, 1], iv[:, :, 1] = k, v
    bg.bg_beam_qk_norm_rope(q, ik[:, :, 1], iv[:, :, 1], base, 3, out, ik, iv, 1, **x["kw"])
    assert torch.equal(ik, sk) and torch.equal(iv, sv)


def test_no_rows():
    import torch
    x = inputs(14, 0, 4, 2, 64)
    q, k, v = split(x)
    e = [torch.empty_like(t.contiguous()) for t in (q, k, v)]
    bg.bg_packed_qk_norm_rope(q, k, v, x["positions"], *e, **x["kw"])


def test_streams_and_graph():
    """Two problems on two streams at once, and a captured call replayed on new inputs."""
    import torch
    xs = [inputs(15, 5000, 16, 8, 128), inputs(16, 777, 14, 2, 64)]
    want = [run(x) for x in xs]
    outs = [[torch.zeros_like(t.contiguous()) for t in split(x)] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for x, o, s in zip(xs, outs, streams):
        bg.bg_packed_qk_norm_rope(*split(x), x["positions"], *o, stream=s, **x["kw"])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))
    x, o = xs[0], outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bg.bg_packed_qk_norm_rope(*split(x), x["positions"], *o, **x["kw"])
    y = inputs(17, 5000, 16, 8, 128)
    x["qkv"].copy_(y["qkv"])
    x["positions"].copy_(y["positions"])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, run(x)))


def test_element_offsets_past_31_bits():
    import torch
    rows, Hq, Hkv, d = (1 << 19) + 5, 30, 1, 128
    assert rows * (Hq + 2 * Hkv) * d > 1 << 31
    x = inputs(18, 40, Hq, Hkv, d)
    big = torch.zeros((rows, (Hq + 2 * Hkv) * d), dtype=torch.bfloat16, device="cuda")
    big[-40:] = x["qkv"]
    pos = torch.zeros((1, rows), dtype=torch.int32, device="cuda")
    pos[:, -40:] = x["positions"]
    y = dict(x, qkv=big, positions=pos)
    o = [torch.empty((rows, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
    bg.bg_packed_qk_norm_rope(*split(y), pos, *o, **x["kw"])
    want = run(x)
    assert all(torch.equal(a[-40:], b) for a, b in zip(o, want)) and (o[0][:-40] == 0).all()
