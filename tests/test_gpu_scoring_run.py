"""A scoring request through the calls as a user strings them together: the prefixes by
bg_packed_prefill_attn, the samples' tokens by bg_shared_prefill_attn over the prefixes' K and V, the last
layer by bg_shared_last_token_attn, and the answers by bg_token_logprobs.  Every call reads what the
one before it left on the device, and is compared with the fp64 oracle on just that."""
import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from oracle import shared as sh
from tests.helpers import from_dev, i32_dev
from tests.test_gpu_logprobs import compare
from tests.test_gpu_shared import assert_close, f64

pytestmark = pytest.mark.gpu

D_MODEL = 256
PREFIX = [150, 0, 33]
GROUPS = [[20, 1, 64], [7, 130], [3, 3, 3, 3]]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


class Model:
    """Two attention layers and a head of random weights: bf16 tensors, products by torch."""

    def __init__(self, Hq, Hkv, d, vocab, softcap):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(31)
        self.Hq, self.Hkv, self.d, self.softcap, self.scale = Hq, Hkv, d, softcap, d ** -0.5

        def w(a, b):
            return (torch.randn((a, b), generator=gen, device="cuda") * a ** -0.5).to(torch.bfloat16)

        self.qkv = [w(D_MODEL, (Hq + 2 * Hkv) * d) for _ in range(2)]
        self.o, self.head = w(Hq * d, D_MODEL), w(Hq * d, vocab)
        self.prefix = torch.randn((sum(PREFIX), D_MODEL), generator=gen, device="cuda").to(torch.bfloat16)
        self.own = torch.randn((sum(map(sum, GROUPS)), D_MODEL), generator=gen, device="cuda").to(torch.bfloat16)

        def cu(x):
            return np.concatenate(([0], np.cumsum(x))).astype(np.int32)

        self.h_cu, self.h_cup = cu([n for g in GROUPS for n in g]), cu(PREFIX)
        self.h_cug = cu([len(g) for g in GROUPS])
        self.cu, self.cup, self.cug = i32_dev(self.h_cu), i32_dev(self.h_cup), i32_dev(self.h_cug)
        self.ends = torch.from_numpy(self.h_cu[1:].astype(np.int64) - 1).cuda()
        self.n, self.mp = int(np.diff(self.h_cu).max()), int(np.diff(self.h_cup).max())
        S, T, P = len(self.h_cu) - 1, int(self.h_cu[-1]), int(self.h_cup[-1])
        self.tokens = torch.randint(vocab, (S,), generator=gen, device="cuda", dtype=torch.int32)
        self.ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
            bg.bg_packed_prefill_workspace_size(len(PREFIX), P, self.mp, Hq, Hkv, d),
            bg.bg_shared_attn_workspace_size(len(GROUPS), S, T, self.n, self.mp, Hq, Hkv, d))]
        self.kept = {}

    def split(self, x, layer):
        y = x @ self.qkv[layer]
        parts = y.split([self.Hq * self.d, self.Hkv * self.d, self.Hkv * self.d], 1)
        return [p.reshape(x.shape[0], h, self.d).contiguous() for p, h in zip(parts, (self.Hq, self.Hkv, self.Hkv))]

    def run(self, planned):
        import torch
        # layer 1: the prefixes by themselves, the samples over them
        pq, pk, pv = self.split(self.prefix, 0)
        q, k, v = self.split(self.own, 0)
        pout, out = torch.empty_like(pq), torch.empty_like(q)
        bg.bg_packed_prefill_attn(pq, pk, pv, self.cup, self.mp, pout, scale=self.scale, workspace=self.ws[0])
        args = (self.cu, self.n, pk, pv, self.cup, self.mp, self.cug)
        kw = dict(scale=self.scale, softcap=self.softcap, workspace=self.ws[1])
        sizes = (self.cu, q.shape[0], self.n, self.cup, pq.shape[0], self.mp, self.cug, self.Hq, self.Hkv, self.d)
        if planned:
            bg.bg_shared_prefill_plan(*sizes, workspace=self.ws[1])
            bg.bg_shared_prefill_attn_planned(q, k, v, *args, out, **kw)
        else:
            bg.bg_shared_prefill_attn(q, k, v, *args, out, **kw)
        # layer 2: K and V of every row, the queries of the samples' last tokens
        _, pk2, pv2 = self.split(self.prefix + pout.flatten(1) @ self.o, 1)
        q2, k2, v2 = self.split(self.own + out.flatten(1) @ self.o, 1)
        ql = q2[self.ends]
        last = torch.empty_like(ql)
        args2 = (self.cu, self.n, pk2, pv2, self.cup, self.mp, self.cug)
        if planned:
            bg.bg_shared_last_token_plan(*sizes, workspace=self.ws[1])
            bg.bg_shared_last_token_attn_planned(ql, k2, v2, *args2, last, **kw)
        else:
            bg.bg_shared_last_token_attn(ql, k2, v2, *args2, last, **kw)
        # the answers
        x = (last.flatten(1) @ self.head) * 4
        S = x.shape[0]
        res = dict(logprob=torch.empty(S, device="cuda"), entropy=torch.empty(S, device="cuda"),
                   top_token=torch.empty((S, 5), dtype=torch.int32, device="cuda"),
                   top_logprob=torch.empty((S, 5), device="cuda"))
        bg.bg_token_logprobs(x, self.tokens, **res)
        self.kept = dict(pq=pq, pk=pk, pv=pv, pout=pout, q=q, k=k, v=v, out=out, ql=ql, pk2=pk2, pv2=pv2, k2=k2, v2=v2,
                         last=last, x=x)
        return res

    def check(self, res):
        import torch
        h = {n: np.ascontiguousarray(t.view(torch.int16).cpu().numpy().view(np.uint16)) for n, t in self.kept.items()}
        # the prefix rows against the oracle of the packed call, by the same bounds as the samples (a
        # request of one sample and no prefix is a packed sequence)
        none = f64(h["pk"])[:0]
        ref = sh.attn(f64(h["pq"]), f64(h["pk"]), f64(h["pv"]), self.h_cup, none, none, np.zeros(len(self.h_cup), int),
                      np.arange(len(self.h_cup)), self.scale)
        assert_close(from_dev(self.kept["pout"]), None, ref, "prefixes")
        for q, k, v, pk, pv, out, last in (("q", "k", "v", "pk", "pv", "out", False),
                                           ("ql", "k2", "v2", "pk2", "pv2", "last", True)):
            ref = sh.attn(f64(h[q]), f64(h[k]), f64(h[v]), self.h_cu, f64(h[pk]), f64(h[pv]), self.h_cup, self.h_cug,
                          self.scale, softcap=self.softcap, last=last)
            assert_close(from_dev(self.kept[out]), None, ref, out, self.softcap)
        compare(res, self.kept["x"], self.tokens.cpu().numpy(), 5, "answers")


@pytest.mark.parametrize("planned", [False, True], ids=["one_call", "planned"])
@pytest.mark.parametrize("heads,softcap", [((16, 8, 128), 0.0), ((14, 2, 64), 30.0), ((4, 4, 64), 0.0)])
def test_scoring_request(heads, softcap, planned):
    m = Model(*heads, 5003, softcap)
    m.check(m.run(planned))


def test_scoring_request_in_one_graph():
    """The whole run captured once and replayed on new inputs in the same buffers."""
    import torch
    m = Model(16, 8, 128, 5003, 0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.run(False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        res = m.run(False)
    for seed in (41, 42):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        m.prefix.copy_(torch.randn(m.prefix.shape, generator=gen, device="cuda"))
        m.own.copy_(torch.randn(m.own.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        m.check(res)


def test_samples_equal_whole_sequences():
    """The samples' rows are the last rows of [prefix ; sample] given whole to bg_packed_prefill_attn:
    both within their bounds of the same exact value."""
    import torch
    m = Model(16, 8, 128, 5003, 0.0)
    m.run(False)
    seqs, at = [], 0
    for r, group in enumerate(GROUPS):
        for n in group:
            seqs.append((slice(m.h_cup[r], m.h_cup[r + 1]), slice(at, at + n)))
            at += n
    full = [torch.cat([torch.cat((m.kept["p" + t][p], m.kept[t][s])) for p, s in seqs]) for t in ("q", "k", "v")]
    lens = [p.stop - p.start + s.stop - s.start for p, s in seqs]
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    out = torch.empty_like(full[0])
    ws = torch.empty(bg.bg_packed_prefill_workspace_size(len(lens), int(cu[-1]), max(lens), 16, 8, 128),
                     dtype=torch.uint8, device="cuda")
    bg.bg_packed_prefill_attn(*full, i32_dev(cu), max(lens), out, scale=m.scale, workspace=ws)
    whole = torch.cat([out[e - (s.stop - s.start):e] for (p, s), e in zip(seqs, cu[1:].tolist())])
    h = {n: np.ascontiguousarray(t.view(torch.int16).cpu().numpy().view(np.uint16)) for n, t in m.kept.items()}
    ref = sh.attn(f64(h["q"]), f64(h["k"]), f64(h["v"]), m.h_cu, f64(h["pk"]), f64(h["pv"]), m.h_cup, m.h_cug, m.scale)
    assert_close(from_dev(whole), None, ref, "whole sequences")
    assert_close(from_dev(m.kept["out"]), None, ref, "samples")
