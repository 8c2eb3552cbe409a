"""GPU parity of bg_token_logprobs (through the C ABI) with the fp64 oracle on the same logits."""
import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from oracle import logprobs as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


def logits(seed, N, V, dtype, banned=0.0, scale=2.5):
    """A torch CPU tensor [N, V] of the type."""
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(0, scale, (N, V)).astype(np.float32)
    if banned:
        x[:, rng.random(V) < banned] = -np.inf
    return torch.from_numpy(x).to(getattr(torch, dtype))


def run(x, tokens, K, dev_status=None, **kw):
    import torch
    N = x.shape[0]
    o = dict(logprob=torch.full((N,), 55.0, device="cuda"), entropy=torch.full((N,), 55.0, device="cuda"))
    if K:
        o.update(top_token=torch.full((N, K), -7, dtype=torch.int32, device="cuda"),
                 top_logprob=torch.full((N, K), 55.0, device="cuda"))
    t = torch.as_tensor(np.asarray(tokens, np.int32)).cuda()
    bg.bg_token_logprobs(x if x.is_cuda else x.cuda(), t, dev_status=dev_status, **o, **kw)
    return o


def compare(o, x, tokens, K, what=""):
    """Tokens are equal.  With c = V / 512 + 64 sequential fp32 additions at most on a term's way into a
    sum (a thread's share and the joins), Z is off by c 2^-24 of itself, its terms by 2^-22 (the
    exponential) and 2^-23 (the exponent's rounding): c 2^-23 + 2^-21 on ln Z.  The entropy's second
    sum has the same relative error of its at most entropy + 1 value; results round once more."""
    lp, H, top, tlp = ol.token_logprobs(x.float().cpu().numpy(), tokens, K)
    c = x.shape[1] / 512 + 64
    e = c * 2.0 ** -23 + 2.0 ** -21

    def close(got, ref, tol, name):
        got = got.double().cpu().numpy()
        fin = np.isfinite(ref)
        assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~fin & ~np.isnan(ref)],
                                                                               ref[~fin & ~np.isnan(ref)]), (what, name)
        err = np.abs(got[fin] - ref[fin])
        assert (err <= np.broadcast_to(tol, ref.shape)[fin]).all(), (what, name, err.max())

    def size(a):
        return np.abs(np.where(np.isfinite(a), a, 0))

    close(o["logprob"], lp, e + 2.0 ** -22 * size(lp), "logprob")
    close(o["entropy"], H, 2 * e * (size(H) + 1) + 2.0 ** -23 * size(H), "entropy")
    if K:
        assert np.array_equal(o["top_token"].cpu().numpy(), top), what
        close(o["top_logprob"], tlp, e + 2.0 ** -22 * size(tlp), "top_logprob")


def check(x, K, what="", seed=1):
    tokens = np.random.default_rng(seed).integers(0, x.shape[1], x.shape[0])
    compare(run(x, tokens, K), x, tokens, K, what)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 33, 512, 1025, 1919, 1927, 2049, 3841, 4097, 8191, 16384, 50001, 65536,
                               151936])
def test_vocabularies(V, dtype):
    for N, K in ((1, 1), (3, min(V, 5)), (5, min(V, 32))):
        check(logits(V + N, N, V, dtype, banned=0.1 if V > 50 else 0.0), K, f"V {V} N {N} K {K}")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("N", [2, 9, 20, 39, 77, 160, 310, 700])
def test_row_counts(N, dtype):
    """Every number of CTAs per row, and more rows than CTAs."""
    check(logits(N, N, 20011, dtype), 20, f"N {N}")


def test_very_long_rows():
    check(logits(5, 2, 1 << 20, "float32"), 32, "1M fp32")
    check(logits(6, 1, 1 << 22, "bfloat16"), 8, "4M bf16")
    check(logits(7, 320, 150001, "float32")[:305], 8, "one CTA per long row")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_ties_and_flat_rows(dtype):
    """Rows of few distinct values: the order is by the smaller token, also where thousands tie."""
    import torch
    x = (logits(8, 6, 30000, "float32") * 0.4).round()
    x[0] = 0.0
    x[1] = -3.5
    x[1, 29999] = 2.0
    x[2, 100:] = x[2].max() + 1
    x[3, ::2] = 0.0
    x[3, 1::2] = -0.0
    check(x.to(getattr(torch, dtype)), 32, "ties")
    check(x[:, :901].to(getattr(torch, dtype)).contiguous(), 7, "short ties")


def test_sorted_and_clustered_rows():
    import torch
    x = torch.sort(logits(9, 4, 60000, "float32"), dim=1).values
    x[1] = x[1].flip(0)
    x[2, 1000:1032] = 50.0 + torch.arange(32.0)      # all of the best in one batch
    x[3, 5::512 * 4] = 40.0 + torch.arange(x[3, 5::2048].numel())     # ... and in one thread
    check(x, 32, "sorted")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_rows_without_a_distribution(dtype):
    """Banned everywhere, NaN, +inf, a single live token, and values at the type's ends."""
    import torch
    x = logits(10, 9, 5000, dtype)
    top = torch.finfo(getattr(torch, dtype)).max
    x[0] = -float("inf")
    x[1, 4321] = float("nan")
    x[2, 17] = float("inf")
    x[3] = -float("inf")
    x[3, 777] = -1.0
    x[4] = -top
    x[5, 4999] = float("nan")
    x[6] = -top
    x[6, 3] = 0.0
    x[7, :] = 1000.0
    check(x, 6, "no distribution")
    check(x[:, :40].contiguous(), 32, "no distribution, short")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strided_and_unaligned_rows(dtype):
    """Rows of a wider buffer, at every alignment of the element."""
    big = logits(11, 7, 9001, dtype).cuda()
    for off in range(0, 9):
        check(big[:, off:off + 8003], 9, f"offset {off}")
    check(big[::2, 3:4000], 9, "every other row")
    check(big[:1, 1:50], 9, "one row")


def test_outputs_are_optional_and_bad_tokens_reported():
    import torch
    x = logits(12, 6, 3000, "float32")
    tok = np.array([0, 2999, -1, 3000, 5, 1 << 30], np.int64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = run(x, tok, 4, dev_status=st)
    assert int(st.item()) == bg.BG_DEVSTAT_TOKEN
    ok = [0, 1, 4]
    assert (o["logprob"].cpu().numpy()[[2, 3, 5]] == 55.0).all()
    compare({n: t[ok] for n, t in o.items()}, x[ok], tok[ok], 4)
    compare({n: t[[2, 3, 5]] for n, t in o.items() if n != "logprob"} | {"logprob": torch.tensor(
        ol.token_logprobs(x[[2, 3, 5]].numpy(), [0, 0, 0], 4)[0])}, x[[2, 3, 5]], [0, 0, 0], 4)
    # one output at a time
    alone = torch.empty(6, device="cuda")
    bg.bg_token_logprobs(x.cuda(), entropy=alone)
    assert torch.equal(alone, o["entropy"])
    t4, l4 = torch.empty((6, 4), dtype=torch.int32, device="cuda"), torch.empty((6, 4), device="cuda")
    bg.bg_token_logprobs(x.cuda(), top_token=t4, top_logprob=l4)
    assert torch.equal(t4, o["top_token"]) and torch.equal(l4, o["top_logprob"])
    check(x, 0, "K 0")


def test_repeats_graph_and_side_stream():
    """Bit-identical repeats, also on another stream and from a captured graph with new logits."""
    import torch
    for N, V in ((3, 40000), (400, 5000)):
        x, y = logits(13, N, V, "bfloat16").cuda(), logits(14, N, V, "bfloat16").cuda()
        tok = np.arange(N) % V
        a, b = run(x, tok, 8), run(y, tok, 8)
        buf = x.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = {n: torch.zeros_like(t) for n, t in a.items()}
        t = torch.as_tensor(tok.astype(np.int32)).cuda()
        torch.cuda.synchronize()
        bg.bg_token_logprobs(buf, t, stream=side, **out)
        side.synchronize()
        assert all(torch.equal(out[n], a[n]) for n in a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bg.bg_token_logprobs(buf, t, **out)
        for src, ref in ((y, b), (x, a)):
            buf.copy_(src)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(out[n], ref[n]) for n in a)


def test_row_offsets_past_32_bits():
    """Rows of a buffer of more than 2^32 elements, whose stride is far above the vocabulary."""
    import torch
    N, V, stride = 4200, 5000, 1 << 20
    assert N * stride > 1 << 32
    buf = torch.empty((N, stride), dtype=torch.bfloat16, device="cuda")
    x = logits(15, N, V, "bfloat16").cuda()
    buf[:, :V] = x
    tok = np.random.default_rng(15).integers(0, V, N)
    a, b = run(x, tok, 8), run(buf[:, :V], tok, 8)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,V", [(330, 30011), (608, 25001), (900, 5003)])
def test_odd_rows_among_many(N, V, dtype):
    """Rows for teams of 8 and of 4 warps: ties, flat rows, banned ones and rows without a distribution
    beside ordinary ones."""
    import torch
    x = logits(16, N, V, dtype)
    x[5] = 0.0
    x[17] = (x[17] * 0.4).round()
    x[100] = -float("inf")
    x[101, V - 1] = float("nan")
    x[200, ::2] = -float("inf")
    x[201, 3] = float("inf")
    x[300] = -torch.finfo(x.dtype).max
    x[N - 1] = torch.sort(x[N - 1]).values
    check(x, 32, f"{N} x {V}")
