"""GPU parity of bg_adjust_logits (through the C ABI) with the fp64 oracle, and its edges: empty and full masks,
values that are not finite, tokens listed twice or outside the vocabulary, strides, bad device data."""
import math

import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from oracle import logits as olg

pytestmark = pytest.mark.gpu

GUARD = 777.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


def i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def packed(lists):
    return i32([t for x in lists for t in x]), i32(np.concatenate(([0], np.cumsum([len(x) for x in lists]))).tolist())


def make(seed, groups, per, V, *, dtype="float32", prompt=20, own=6, bias=5, masks=4, allowed=0.3):
    """Host lists (for the oracle) and device tensors (for the call) of one problem."""
    import torch
    rng = np.random.default_rng(seed)
    N = groups * per
    x = torch.from_numpy((rng.standard_normal((N, V)) * 3).astype(np.float32)).to(getattr(torch, dtype)).cuda()
    h, t = dict(logits=x.double().cpu().numpy(), per=per), dict(rows_per_group=per)

    def some(n):
        return rng.integers(0, V, n).tolist()

    if prompt:
        h["prompts"] = [some(int(rng.integers(0, prompt + 1))) for _ in range(groups)]
        t["prompt_tokens"], t["cu_prompt"] = packed(h["prompts"])
    if own:
        lens = rng.integers(0, own + 1, N)
        tokens = rng.integers(0, max(1, min(V, 2 * own)), (N, own))        # repeated ones among them
        h["own"] = [tokens[i, :lens[i]].tolist() for i in range(N)]
        t.update(own_tokens=i32(tokens.tolist()).view(N, own), own_lens=i32(lens.tolist()))
    for name, lo, hi in (("repetition", 0.7, 1.6), ("frequency", -0.2, 0.8), ("presence", -0.5, 1.0)):
        v = rng.uniform(lo, hi, groups).astype(np.float32)
        h[name], t[name] = v, torch.from_numpy(v).cuda()
    if bias:
        h["biases"] = [[(tk, np.float32(rng.normal())) for tk in some(int(rng.integers(0, bias + 1)))] for _ in range(groups)]
        t["bias_tokens"], t["cu_bias"] = packed([[b[0] for b in g] for g in h["biases"]])
        t["bias_values"] = torch.tensor([float(b[1]) for g in h["biases"] for b in g], device="cuda")
    if masks:
        bits = rng.random((masks, V)) < allowed
        if masks > 1:
            bits[1] = False
        if masks > 2:
            bits[2] = True
        index = rng.integers(-1, masks, N)
        h["masks"] = [None if m < 0 else set(np.flatnonzero(bits[m]).tolist()) for m in index]
        t.update(mask=words_of(bits), mask_index=i32(index.tolist()))
    return h, x, t


def words_of(bits):
    """bool [M,V] to int32 words; the bits past V are set."""
    import torch
    M, V = bits.shape
    full = np.ones((M, (V + 31) // 32 * 32), np.uint8)
    full[:, :V] = bits
    w = np.packbits(full.reshape(M, -1, 32), axis=-1, bitorder="little").view(np.uint32)[..., 0]
    return torch.from_numpy(np.ascontiguousarray(w).view(np.int32)).cuda()


def assert_close(got, ref, bf16):
    """At most five roundings of fp32 (2^-24 each, of no more than the magnitudes that were added), and one to bf16
    (2^-8); what is masked is -inf exactly."""
    out, size = ref
    got = got.double().cpu().numpy()
    fine = np.isfinite(out)
    assert np.array_equal(got[~fine], out[~fine], equal_nan=True)
    e = 5 * 2.0 ** -24 * size
    tol = e + (2.0 ** -8 * (np.abs(out) + e) if bf16 else 0.0)
    err = np.abs(got[fine] - out[fine])
    assert (err <= tol[fine]).all(), (err - tol[fine]).max()


def check(h, x, t, *, out_dtype="float32", **kw):
    import torch
    dt = getattr(torch, out_dtype)
    N, V = x.shape
    full = torch.full((N * V + 64,), GUARD, dtype=dt, device="cuda")
    out = full[:N * V].view(N, V)
    st = i32([0])
    bg.bg_adjust_logits(x, out, dev_status=st, **t, **kw)
    assert int(st.item()) == 0 and (full[N * V:] == GUARD).all()
    assert_close(out, olg.adjust(**h), out_dtype == "bfloat16")
    return out


TYPES = [("float32", "float32"), ("bfloat16", "float32"), ("bfloat16", "bfloat16")]


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 100, 1000, 1024, 1025, 4104, 8192, 8193, 20000, 50001])
def test_parity(V, types):
    check(*make(V, 3, 4, V, dtype=types[0]), out_dtype=types[1])


@pytest.mark.parametrize("without", [("prompt",), ("own",), ("bias",), ("masks",), ("prompt", "own", "bias"),
                                     ("prompt", "own", "masks"), ("prompt", "own", "bias", "masks")], ids="-".join)
@pytest.mark.parametrize("V", [1000, 9001])
def test_parts_left_out(V, without):
    check(*make(2, 2, 3, V, **{n: 0 for n in without}))


@pytest.mark.parametrize("none", ["repetition", "frequency", "presence"])
def test_penalties_left_out(none):
    h, x, t = make(3, 3, 2, 3000)
    h[none] = t[none] = None
    check(h, x, t)


def test_untouched_logits_keep_their_bits():
    import torch
    for types in TYPES:
        h, x, t = make(4, 2, 2, 5000, dtype=types[0], masks=0)
        out = check(h, x, t, out_dtype=types[1])
        same = np.ones((4, 5000), bool)
        for i in range(4):
            same[i, h["prompts"][i // 2] + h["own"][i] + [b[0] for b in h["biases"][i // 2]]] = False
        same = torch.from_numpy(same).cuda()
        assert torch.equal(out[same], x[same].to(out.dtype))


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_many_rows_of_a_group(types):
    """More rows than one CTA takes, and groups of one row."""
    check(*make(5, 2, 150, 9000, dtype=types[0], prompt=300, own=30, bias=100), out_dtype=types[1])
    check(*make(6, 301, 1, 1500, dtype=types[0]), out_dtype=types[1])


def test_long_lists():
    check(*make(7, 2, 3, 30000, prompt=20000, own=5000, bias=bg.BG_MAX_BIAS))


def test_counts_to_the_limit():
    """65536 times the same token, in every row."""
    import torch
    n = bg.BG_MAX_SEQLEN
    x = torch.zeros((3, 64), device="cuda")
    own = torch.full((3, n), 7, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    bg.bg_adjust_logits(x, out, rows_per_group=3, own_tokens=own, frequency=torch.tensor([0.5], device="cuda"),
                        presence=torch.tensor([1.0], device="cuda"))
    want = torch.zeros_like(x)
    want[:, 7] = -(0.5 * n + 1)
    assert torch.equal(out, want)


def test_own_tokens_without_lengths():
    h, x, t = make(8, 2, 2, 3000, own=9)
    h["own"] = t["own_tokens"].tolist()
    t["own_lens"] = None
    check(h, x, t)


def test_mask_of_each_row():
    """Without an index row i has mask i; words beyond the vocabulary's do not matter."""
    import torch
    rng = np.random.default_rng(9)
    h, x, t = make(9, 2, 3, 1003, masks=0)
    bits = rng.random((6, 1003)) < 0.5
    h["masks"] = [set(np.flatnonzero(b).tolist()) for b in bits]
    w = words_of(bits)
    check(h, x, dict(t, mask=w))
    check(h, x, dict(t, mask=torch.cat((w, torch.full((6, 3), -1, dtype=torch.int32, device="cuda")), 1)))
    if hasattr(torch, "uint32"):
        check(h, x, dict(t, mask=w.view(torch.uint32)))


@pytest.mark.parametrize("V", [64, 2051])
def test_masks_of_all_or_none(V):
    import torch
    h, x, t = make(10, 1, 3, V, masks=0)
    bits = np.array([[False] * V, [True] * V, [False] * V])
    bits[2, V - 1] = True
    h["masks"] = [set(np.flatnonzero(b).tolist()) for b in bits]
    out = check(h, x, dict(t, mask=words_of(bits)))
    assert torch.isneginf(out[0]).all() and torch.isneginf(out[2, :-1]).all()


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_values_that_are_not_finite(types):
    """In masked places they vanish, elsewhere they go through the formula; neighbours do not notice."""
    import torch
    h, x, t = make(11, 2, 2, 400, dtype=types[0], masks=1, allowed=0.5)
    t["mask_index"].zero_()
    words = t["mask"].cpu().numpy().view(np.uint32)[0]
    allowed = [v for v in range(400) if words[v // 32] >> (v % 32) & 1]
    banned = [v for v in range(400) if v not in set(allowed)]
    h["masks"] = [set(allowed)] * 4
    low = torch.finfo(x.dtype).min
    for i, v in enumerate((math.nan, math.inf, -math.inf, low)):
        x[i % 4, banned[3 * i]] = v
        x[i % 4, allowed[3 * i]] = v
    h["logits"] = x.double().cpu().numpy()
    h["repetition"] = np.full(2, 1.0, np.float32)         # the lowest value times a penalty would overflow
    t["repetition"] = torch.ones(2, device="cuda")
    for name in ("frequency", "presence"):
        h[name], t[name] = None, None
    h["biases"] = [[(allowed[40], np.float32(1.5))]] * 2
    t["bias_tokens"], t["cu_bias"] = packed([[allowed[40]]] * 2)
    t["bias_values"] = torch.tensor([1.5, 1.5], device="cuda")
    check(h, x, t, out_dtype=types[1])


def test_infinite_biases_and_overflow():
    import torch
    x = torch.tensor([[1.0, 2.0, 3.0e38, -3.0e38]], device="cuda")
    out = torch.empty_like(x)
    bg.bg_adjust_logits(x, out, own_tokens=i32([[2, 3]]), repetition=torch.tensor([0.5], device="cuda"),
                        bias_tokens=i32([0, 3]), cu_bias=i32([0, 2]), bias_values=torch.tensor([-math.inf, 1.0], device="cuda"))
    assert out.tolist()[0][:3] == [-math.inf, 2.0, math.inf] and out[0, 3] == -1.5e38


def test_tokens_listed_twice():
    """The last bias counts, wherever the earlier ones are; a prompt's token counts once."""
    import torch
    V = 300
    x = torch.zeros((1, V), device="cuda") + 2
    n = 1000
    tokens = [5] * n + [7, 5, 7]
    values = list(range(n)) + [1.0, -3.0, 0.25]
    out = torch.empty_like(x)
    bg.bg_adjust_logits(x, out, prompt_tokens=i32([9] * 500 + [5]), cu_prompt=i32([0, 501]),
                        repetition=torch.tensor([2.0], device="cuda"), bias_tokens=i32(tokens), cu_bias=i32([0, n + 3]),
                        bias_values=torch.tensor(values, dtype=torch.float32, device="cuda"))
    want = torch.full((1, V), 2.0, device="cuda")
    want[0, 5], want[0, 7], want[0, 9] = 1.0 - 3.0, 2.25, 1.0
    assert torch.equal(out, want)


def test_tokens_outside_the_vocabulary():
    import torch
    h, x, t = make(12, 2, 2, 500)
    want = torch.empty_like(x)
    bg.bg_adjust_logits(x, want, **t)
    for name in ("prompt_tokens", "own_tokens", "bias_tokens"):
        u = dict(t)
        if name == "own_tokens":
            wide = torch.cat((i32([[-1], [500], [1 << 30], [-(1 << 31)]]), t["own_tokens"]), 1)
            u.update(own_tokens=wide.contiguous(), own_lens=t["own_lens"] + 1)
        else:
            cu = name.replace("tokens", "").strip("_")
            key = "cu_" + cu
            a, b = (t[name][t[key][g]:t[key][g + 1]] for g in range(2))
            bad = i32([-7, 500])
            u[name] = torch.cat((bad, a, b, bad))
            u[key] = t[key] + i32([0, 2, 4])
            if name == "bias_tokens":
                va, vb = (t["bias_values"][t[key][g]:t[key][g + 1]] for g in range(2))
                z = torch.full((2,), 9.0, device="cuda")
                u["bias_values"] = torch.cat((z, va, vb, z))
        out, st = torch.empty_like(x), i32([0])
        bg.bg_adjust_logits(x, out, dev_status=st, **u)
        assert int(st.item()) == bg.BG_DEVSTAT_TOKEN, name
        assert torch.equal(out, want), name
        bg.bg_adjust_logits(x, out.zero_(), **u)                 # without a status word
        assert torch.equal(out, want), name


def test_bad_offsets_lengths_and_masks():
    """The group or row is left as it was and reported; the others are written."""
    import torch
    h, x, t = make(13, 3, 2, 900, prompt=9, bias=4, own=5)
    want = torch.empty_like(x)
    bg.bg_adjust_logits(x, want, **t)
    total, tb = t["prompt_tokens"].numel(), t["bias_tokens"].numel()
    cases = [("cu_prompt", [0, 3, 2, total], {1}, bg.BG_DEVSTAT_CU_PROMPT), ("cu_prompt", [0, 0, total + 1, total], {1, 2},
             bg.BG_DEVSTAT_CU_PROMPT), ("cu_prompt", [-1, 0, 0, total], {0}, bg.BG_DEVSTAT_CU_PROMPT),
             ("cu_prompt", [0, 0, 0, total - 1], {2}, bg.BG_DEVSTAT_CU_PROMPT), ("cu_bias", [0, tb, 0, tb], {1}, bg.BG_DEVSTAT_BIAS),
             ("cu_bias", [1, 1, 1, tb], {0}, bg.BG_DEVSTAT_BIAS)]
    for name, bad, groups, bit in cases:
        out, st = torch.full_like(x, GUARD), i32([0])
        bg.bg_adjust_logits(x, out, dev_status=st, **dict(t, **{name: i32(bad)}))
        assert int(st.item()) == bit, (name, bad)
        assert all((out[2 * g:2 * g + 2] == GUARD).all() == (g in groups) for g in range(3)), (name, bad)
    for name, row, value, bit in (("own_lens", 3, 6, bg.BG_DEVSTAT_SEQ_TOO_LONG), ("own_lens", 0, -1, bg.BG_DEVSTAT_SEQ_TOO_LONG),
                                  ("mask_index", 5, 4, bg.BG_DEVSTAT_MASK), ("mask_index", 2, -2, bg.BG_DEVSTAT_MASK)):
        bad = t[name].clone()
        bad[row] = value
        out, st = torch.full_like(x, GUARD), i32([0])
        bg.bg_adjust_logits(x, out, dev_status=st, **dict(t, **{name: bad}))
        assert int(st.item()) == bit
        rest = [i for i in range(6) if i != row]
        assert (out[row] == GUARD).all() and torch.equal(out[rest], want[rest])


def test_too_many_biases():
    import torch
    n = bg.BG_MAX_BIAS + 1
    x = torch.zeros((2, 100), device="cuda")
    out, st = torch.full_like(x, GUARD), i32([0])
    bg.bg_adjust_logits(x, out, bias_tokens=i32([3] * n + [4]), bias_values=torch.ones(n + 1, device="cuda"),
                        cu_bias=i32([0, n, n + 1]), dev_status=st)
    assert int(st.item()) == bg.BG_DEVSTAT_BIAS and (out[0] == GUARD).all() and out[1, 4] == 1 and out[1].sum() == 1


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("pad_in,pad_out,at", [(3, 0, 0), (0, 5, 0), (8, 16, 8), (7, 7, 1)])
def test_strides_and_alignment(pad_in, pad_out, at, types):
    import torch
    V = 2043 if pad_in == 3 else 2048
    h, x, t = make(14, 2, 5, V, dtype=types[0])
    dt = getattr(torch, types[1])
    src = torch.full((10, V + pad_in + at), GUARD, dtype=x.dtype, device="cuda")
    dst = torch.full((10, V + pad_out + at), GUARD, dtype=dt, device="cuda")
    src[:, at:at + V] = x
    bg.bg_adjust_logits(src[:, at:at + V], dst[:, at:at + V], **t)
    assert_close(dst[:, at:at + V], olg.adjust(**h), types[1] == "bfloat16")
    assert (dst[:, :at] == GUARD).all() and (dst[:, at + V:] == GUARD).all()


@pytest.mark.parametrize("V", [1001, 9008])
def test_in_place(V):
    import torch
    for dtype in ("float32", "bfloat16"):
        h, x, t = make(15, 3, 7, V, dtype=dtype)
        want = torch.empty_like(x)
        bg.bg_adjust_logits(x, want, **t)
        bg.bg_adjust_logits(x, x, **t)
        assert torch.equal(x, want)


def test_no_rows_and_empty_lists():
    import torch
    e = torch.empty((0, 50), device="cuda")
    bg.bg_adjust_logits(e, torch.empty_like(e), rows_per_group=4)
    x = torch.randn((4, 50), device="cuda")
    out = torch.empty_like(x)
    z = torch.zeros(5, dtype=torch.int32, device="cuda")
    bg.bg_adjust_logits(x, out, prompt_tokens=i32([]), cu_prompt=z, own_tokens=torch.empty((4, 0), dtype=torch.int32, device="cuda"),
                        own_lens=z[:4], bias_tokens=i32([]), bias_values=torch.empty(0, device="cuda"), cu_bias=z,
                        repetition=torch.full((4,), 2.0, device="cuda"))
    assert torch.equal(out, x)


def test_streams_graph_and_repeatability():
    import torch
    ps = [make(16, 4, 20, 30000), make(17, 7, 3, 5001, dtype="bfloat16")]
    want, outs = [], []
    for _, x, t in ps:
        w = torch.empty(x.shape, device="cuda")
        bg.bg_adjust_logits(x, w, **t)
        want.append(w)
        outs.append(torch.zeros_like(w))
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(3):
        for (_, x, t), o, s in zip(ps, outs, streams):
            bg.bg_adjust_logits(x, o, stream=s, **t)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    (_, x, t), o = ps[0], outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bg.bg_adjust_logits(x, o, **t)
    x.add_(1)
    t["mask_index"].fill_(-1)
    graph.replay()
    bg.bg_adjust_logits(x, want[0], **t)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0])


def test_element_offsets_past_31_bits():
    import torch
    V = 1 << 22
    rows = 515
    assert rows * V > 1 << 31
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device="cuda")
    x[-1, -8:] = 1
    own = torch.full((rows, 1), V - 1, dtype=torch.int32, device="cuda")
    bg.bg_adjust_logits(x, x, rows_per_group=rows, own_tokens=own, presence=torch.tensor([3.0], device="cuda"))
    assert x[-1, -9:].tolist() == [0.0] + [1.0] * 7 + [-2.0] and (x[:-1, -1] == -3).all() and (x[:, :-8] == 0).all()


@pytest.mark.parametrize("own", [3, 40], ids=["few", "many"])
@pytest.mark.parametrize("V", [70, 5000, 4096 * 3 + 5])
def test_more_rows_than_a_cta_takes(V, own):
    """Groups of many rows, each with a mask, list and history of its own, and rows that are refused among them."""
    import torch
    h, x, t = make(20, 3, 67, V, own=own, prompt=30, bias=9, masks=7)
    want = check(h, x, t)
    bad = t["own_lens"].clone()
    bad[[0, 1, 65, 66, 67, 200]] = own + 1
    out, st = torch.full_like(x, GUARD), i32([0])
    bg.bg_adjust_logits(x, out, dev_status=st, **dict(t, own_lens=bad))
    assert int(st.item()) == bg.BG_DEVSTAT_SEQ_TOO_LONG
    ok = (bad <= own).nonzero()[:, 0]
    assert torch.equal(out[ok], want[ok]) and (out[bad > own] == GUARD).all()


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_dense_lists(types):
    """Nearly every token of the first blocks is listed, as a vocabulary's frequent tokens are."""
    import torch
    rng = np.random.default_rng(21)
    V, N = 9000, 6
    h, x, t = make(21, 2, 3, V, dtype=types[0], prompt=0, own=0, bias=0, masks=3, allowed=0.9)
    h["prompts"] = [rng.integers(0, 1500, 6000).tolist() for _ in range(2)]
    t["prompt_tokens"], t["cu_prompt"] = packed(h["prompts"])
    tokens = rng.integers(0, 2500, (N, 3000))
    h["own"], t["own_tokens"] = tokens.tolist(), i32(tokens.tolist())
    h["biases"] = [[(int(k), np.float32(rng.normal())) for k in rng.integers(0, 1200, 2000)] for _ in range(2)]
    t["bias_tokens"], t["cu_bias"] = packed([[b[0] for b in g] for g in h["biases"]])
    t["bias_values"] = torch.tensor([float(b[1]) for g in h["biases"] for b in g], device="cuda")
    check(h, x, t, out_dtype=types[1])
    if types[0] == types[1]:
        want = torch.empty_like(x)
        bg.bg_adjust_logits(x, want, **t)
        bg.bg_adjust_logits(x, x, **t)
        assert torch.equal(x, want)
