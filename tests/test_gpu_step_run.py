"""A decode step and a verify step through the calls as a user strings them together; every call reads what the one
before it left on the device, and is compared with the fp64 oracle on just that.

Decode: projection -> bg_beam_qk_norm_rope -> bg_beam_decode_step -> head -> bg_adjust_logits (a tree of allowed
identifiers) -> bg_beam_select, three steps.  Verify: projection -> bg_packed_qk_norm_rope at the nodes' depths ->
bg_tree_attn over the cached prompt, two layers with one plan -> head -> bg_adjust_logits in place -> bg_token_logprobs."""
import numpy as np
import pytest

import oracle
from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from oracle import logits as olg
from oracle import logprobs as olp
from oracle import rope as orp
from oracle import tree as otr
from tests import test_gpu_logits as tl
from tests import test_gpu_rope as tr
from tests.helpers import assert_parity, bits_from_dev, from_dev, i32_dev
from tests.test_gpu_select import SCORE_TOL
from tests.test_gpu_shared import assert_close

pytestmark = pytest.mark.gpu

D_MODEL, VOCAB, STEPS = 256, 1000, 3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


class Model:
    def __init__(self, Hq, Hkv, d, seed=5):
        import torch
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.d = Hq, Hkv, d

        def w(a, b):
            return (torch.randn((a, b), generator=self.gen, device="cuda") * a ** -0.5).bfloat16()

        self.qkv, self.o, self.head = w(D_MODEL, (Hq + 2 * Hkv) * d), w(Hq * d, D_MODEL), w(D_MODEL, VOCAB)
        self.embed = torch.randn((VOCAB, D_MODEL), generator=self.gen, device="cuda").bfloat16()
        self.kw = dict(inv_freq=tr.frequencies(d // 2), q_weight=(1 + 0.2 * torch.randn(d, generator=self.gen, device="cuda")).bfloat16(),
                       k_weight=(1 + 0.2 * torch.randn(d, generator=self.gen, device="cuda")).bfloat16())

    def split(self, x):
        y = x @ self.qkv
        q, k, v = y.split((self.Hq * self.d, self.Hkv * self.d, self.Hkv * self.d), -1)
        return q.unflatten(-1, (self.Hq, self.d)), k.unflatten(-1, (self.Hkv, self.d)), v.unflatten(-1, (self.Hkv, self.d))

    def turned(self, q, which, pos):
        w = tr.f64(self.kw[which])
        return orp.norm_rotate(tr.f64(q), w, 1e-6, 0.0, pos.cpu().numpy(), tr.f64(self.kw["inv_freq"]))

    def prompt(self, lengths):
        """K and V of the prompts, rotated in place by the packed call."""
        import torch
        x = self.embed[torch.randint(VOCAB, (sum(lengths),), generator=self.gen, device="cuda")]
        q, k, v = (t.contiguous() for t in self.split(x))
        pos = i32_dev(np.concatenate([np.arange(n) for n in lengths]))
        raw = k.clone()
        bg.bg_packed_qk_norm_rope(q, k, v, pos, q, k, v, **self.kw)
        tr.assert_close(k, self.turned(raw, "k_weight", pos[None]))
        return k, v


@pytest.mark.parametrize("heads", [(16, 8, 128), (14, 2, 64)], ids=lambda h: "h%d_%d_d%d" % h)
def test_constrained_beam_search(heads):
    import torch
    m = Model(*heads)
    Hq, Hkv, d = heads
    R, W = 2, 24
    lengths = [70, 33]
    cup = i32_dev(np.concatenate(([0], np.cumsum(lengths))))
    pk, pv = m.prompt(lengths)
    base = i32_dev(np.array(lengths))
    prompt_tokens = torch.randint(VOCAB, (sum(lengths),), generator=m.gen, device="cuda", dtype=torch.int32)
    # identifiers: after a token t the tokens t * 7 + 1 .. + 40 (modulo) may follow; mask VOCAB: the first step, and one
    # state that leaves nothing
    bits = np.zeros((VOCAB + 2, VOCAB), bool)
    for t in range(VOCAB):
        bits[t, (t * 7 + 1 + np.arange(40)) % VOCAB] = True
    bits[VOCAB, ::3] = True
    mask = tl.words_of(bits)
    rep = torch.tensor([1.3, 0.8], device="cuda")

    own = torch.zeros((R, W, STEPS), dtype=torch.int32, device="cuda")
    sk, sv = ([torch.zeros((R, W, STEPS, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2))
    ws = torch.empty(bg.bg_beam_select_workspace_size(R, W, VOCAB), dtype=torch.uint8, device="cuda")
    cum = torch.full((R, W), -float("inf"), device="cuda")
    cum[:, 0] = 0
    parent = torch.zeros((R, W), dtype=torch.int32, device="cuda")
    tokens = torch.full((R, W), 1, dtype=torch.int32, device="cuda")
    hist = oracle.BeamHistory(R, W)
    for step in range(STEPS):
        x = m.embed[tokens.long()]                                       # [R, W, D]
        q, k, v = m.split(x)
        qo = torch.empty((R, W, Hq, d), dtype=torch.bfloat16, device="cuda")
        nk, nv = (torch.empty((R, W, 1, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        bg.bg_beam_qk_norm_rope(q, k, v, base, step, qo, nk, nv, 0, **m.kw)
        pos = (base + step).repeat_interleave(W)[None]
        tr.assert_close(qo.flatten(0, 1), m.turned(q.flatten(0, 1), "q_weight", pos))
        tr.assert_close(nk[:, :, 0].flatten(0, 1), m.turned(k.flatten(0, 1), "k_weight", pos))
        src, dst = step % 2, 1 - step % 2
        out = torch.empty_like(qo)
        bg.bg_beam_decode_step(qo, pk, pv, cup, max(lengths), sk[src], sv[src], parent, nk[:, :, 0], nv[:, :, 0], sk[dst], sv[dst],
                               step + 1, out)
        hist.step(parent.cpu().numpy(), bits_from_dev(nk[:, :, 0]), bits_from_dev(nv[:, :, 0]))
        hk, hv = hist.materialise(Hkv, d)
        assert_parity(from_dev(out), oracle.decode(bits_from_dev(qo), bits_from_dev(pk), bits_from_dev(pv), cup.cpu().numpy(),
                                                   hk, hv, d ** -0.5), f"decode step {step}")
        logits = ((out.flatten(2) @ m.o) @ m.head).float() * 4
        adj = torch.empty_like(logits)
        index = torch.full((R, W), VOCAB, dtype=torch.int32, device="cuda") if step == 0 else tokens.clone()
        if step == 1:
            index[1, 3] = VOCAB + 1                                      # a beam that no identifier continues
        kw = dict(rows_per_group=W, prompt_tokens=prompt_tokens, cu_prompt=cup, repetition=rep, mask=mask, mask_index=index.flatten(),
                  own_tokens=own.flatten(0, 1), own_lens=torch.full((R * W,), step, dtype=torch.int32, device="cuda"))
        bg.bg_adjust_logits(logits.flatten(0, 1), adj.flatten(0, 1), **kw)
        c, o, idx = cup.cpu().numpy(), own.flatten(0, 1).cpu().numpy(), index.flatten().cpu().numpy()
        tl.assert_close(adj.flatten(0, 1), olg.adjust(
            tr.f64(logits.flatten(0, 1)), W, prompts=[prompt_tokens[c[r]:c[r + 1]].tolist() for r in range(R)],
            own=[o[i, :step].tolist() for i in range(R * W)], repetition=rep.cpu().numpy(),
            masks=[set(np.flatnonzero(bits[i]).tolist()) for i in idx]), False)
        new_tok, new_par = torch.empty_like(tokens), torch.empty_like(parent)
        score = torch.empty_like(cum)
        bg.bg_beam_select(adj, cum, new_tok, new_par, score, workspace=ws)
        # every kept candidate is allowed, its score is its parent's plus its log-probability, and none is better
        a = adj.double().cpu().numpy()
        top = a.max(-1, keepdims=True)
        with np.errstate(invalid="ignore", divide="ignore"):
            lp = a - top - np.log(np.exp(a - top).sum(-1, keepdims=True))
        lp[~np.isfinite(a)] = -np.inf
        s = cum.double().cpu().numpy()[:, :, None] + lp
        t, pr, sc = new_tok.cpu().numpy(), new_par.cpu().numpy(), score.double().cpu().numpy()
        for r in range(R):
            kept = s[r, pr[r], t[r]]
            assert np.isfinite(kept).all() and np.abs(sc[r] - kept).max() <= SCORE_TOL
            assert np.abs(kept - np.sort(s[r].ravel())[::-1][:W]).max() <= SCORE_TOL
            assert all(bits[idx[r * W + b]][v] for b, v in zip(pr[r], t[r]))
            if step == 1 and r == 1:
                assert 3 not in pr[r]
        # the next step's beams
        own = own.gather(1, new_par.long()[:, :, None].expand(-1, -1, STEPS)).contiguous()
        own[:, :, step] = new_tok
        tokens, parent, cum = new_tok, new_par, score


def test_beams_with_nothing_left_are_dead():
    """bg_beam_select on rows that a mask has emptied: -inf scores, behind every live candidate."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    for W, V in ((5, 300), (150, 4001)):
        x = torch.randn((2, W, V), generator=gen, device="cuda")
        x[0, 1:] = -float("inf")
        x[0, 0, 3:] = -float("inf")
        x[1, 2] = -float("inf")
        cum = torch.zeros((2, W), device="cuda")
        tok, par = (torch.empty((2, W), dtype=torch.int32, device="cuda") for _ in range(2))
        sc = torch.empty((2, W), device="cuda")
        ws = torch.empty(bg.bg_beam_select_workspace_size(2, W, V), dtype=torch.uint8, device="cuda")
        bg.bg_beam_select(x, cum, tok, par, sc, workspace=ws)
        assert sorted(tok[0, :3].tolist()) == [0, 1, 2] and (par[0, :3] == 0).all() and sc[0, :3].isfinite().all()
        assert torch.isneginf(sc[0, 3:]).all()
        assert sc[1].isfinite().all() and 2 not in par[1].tolist()
        assert all((0 <= t).all() and (t < n).all() for t, n in ((tok, V), (par, W)))


@pytest.mark.parametrize("heads", [(16, 8, 128), (14, 2, 64)], ids=lambda h: "h%d_%d_d%d" % h)
def test_new_tokens_straight_into_the_suffix(heads):
    """Reorder without an append, K and V of the new tokens into their slot, attention: what bg_beam_decode_step gives
    with new_k and new_v, bit for bit."""
    import torch
    m = Model(*heads, seed=6)
    Hq, Hkv, d = heads
    R, W, slots = 3, 33, 4
    lengths = [40, 0, 129]
    cup = i32_dev(np.concatenate(([0], np.cumsum(lengths))))
    pk, pv = m.prompt(lengths)
    base = i32_dev(np.array(lengths))
    src = [torch.randn((R, W, slots, Hkv, d), generator=m.gen, device="cuda").bfloat16() for _ in range(2)]
    for t in (1, 3):
        parent = torch.randint(W, (R, W), generator=m.gen, device="cuda", dtype=torch.int32)
        x = m.embed[torch.randint(VOCAB, (R, W), generator=m.gen, device="cuda")]
        q, k, v = m.split(x)
        nk, nv = (torch.empty((R, W, 1, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q1, q2, o1, o2 = (torch.empty((R, W, Hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(4))
        a, b = ([torch.zeros_like(s) for s in src] for _ in range(2))
        bg.bg_beam_qk_norm_rope(q, k, v, base, t - 1, q1, nk, nv, 0, **m.kw)
        bg.bg_beam_decode_step(q1, pk, pv, cup, max(lengths), *src, parent, nk[:, :, 0], nv[:, :, 0], *a, t, o1)
        bg.bg_beam_suffix_reorder(*src, *b, parent, t - 1)
        bg.bg_beam_qk_norm_rope(q, k, v, base, t - 1, q2, *b, t - 1, **m.kw)
        bg.bg_beam_decode_attn(q2, pk, pv, cup, max(lengths), *b, t, o2)
        assert torch.equal(q1, q2) and torch.equal(o1, o2) and all(torch.equal(s, u) for s, u in zip(a, b))


class Verify:
    """Two layers of a verify step; the buffers stay, so that the whole step can be captured."""

    def __init__(self, heads, softcap):
        import torch
        self.m = m = Model(*heads, seed=8)
        self.softcap = softcap
        Hq, Hkv, d = heads
        self.lengths, self.nodes = [300, 0, 45], [26, 7, 40]
        self.cu, self.cup = (i32_dev(np.concatenate(([0], np.cumsum(n)))) for n in (self.nodes, self.lengths))
        rng = np.random.default_rng(4)
        self.h_parent = np.array([int(rng.integers(max(-1, i - 5), i)) if i else -1 for n in self.nodes for i in range(n)], np.int32)
        depth = []
        for n in self.nodes:
            a = len(depth)
            for i in range(n):
                depth.append(depth[a + self.h_parent[a + i]] + 1 if self.h_parent[a + i] >= 0 else 0)
        self.depth = np.array(depth)
        start = np.repeat(self.lengths, self.nodes)
        self.pos, self.parent = i32_dev(start + self.depth), i32_dev(self.h_parent)
        T = sum(self.nodes)
        self.caches = [m.prompt(self.lengths) for _ in range(2)]
        self.tokens = torch.randint(VOCAB, (T,), generator=m.gen, device="cuda", dtype=torch.int32)
        self.prompt_tokens = torch.randint(VOCAB, (sum(self.lengths),), generator=m.gen, device="cuda", dtype=torch.int32)
        # each node's own tokens: the path to it
        own, lens, a = np.zeros((T, max(self.nodes)), np.int64), np.zeros(T, np.int64), 0
        tok = self.tokens.cpu().numpy()
        self.paths = []
        for n in self.nodes:
            for i in range(n):
                p = [a + j for j in otr.path(self.h_parent[a:a + n], i)]
                own[a + i, :len(p)], lens[a + i] = tok[p], len(p)
                self.paths.append(tok[p].tolist())
            a += n
        self.own, self.lens = i32_dev(own), i32_dev(lens)
        self.group = np.repeat(np.arange(3), self.nodes)
        self.freq = torch.rand(T, generator=m.gen, device="cuda")
        self.ws = torch.empty(bg.bg_tree_attn_workspace_size(3, T, max(self.nodes), max(self.lengths), Hq, Hkv, d),
                              dtype=torch.uint8, device="cuda")
        self.res = dict(logprob=torch.empty(T, device="cuda"), entropy=torch.empty(T, device="cuda"),
                        top_token=torch.empty((T, 4), dtype=torch.int32, device="cuda"), top_logprob=torch.empty((T, 4), device="cuda"))

    def run(self):
        import torch
        m = self.m
        x = m.embed[self.tokens.long()]
        bg.bg_tree_plan(self.parent, self.cu, max(self.nodes), self.cup, sum(self.lengths), max(self.lengths), m.Hq, m.Hkv, m.d,
                        workspace=self.ws)
        self.kept = []
        for pk, pv in self.caches:
            raw = m.split(x)
            q, k, v = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in raw)
            bg.bg_packed_qk_norm_rope(*raw, self.pos, q, k, v, **m.kw)
            out = torch.empty_like(q)
            bg.bg_tree_attn_planned(q, k, v, self.parent, self.cu, max(self.nodes), pk, pv, self.cup, max(self.lengths), out,
                                    softcap=self.softcap, workspace=self.ws)
            self.kept.append((raw, q, k, v, out))
            x = x + out.flatten(1) @ m.o
        self.raw_logits = (x @ m.head) * 3
        self.logits = self.raw_logits.clone()
        bg.bg_adjust_logits(self.logits, self.logits, own_tokens=self.own, own_lens=self.lens, frequency=self.freq)
        bg.bg_token_logprobs(self.logits, self.tokens, **self.res)
        return self.res

    def check(self):
        m = self.m
        for (raw, q, k, v, out), (pk, pv) in zip(self.kept, self.caches):
            tr.assert_close(q, m.turned(raw[0], "q_weight", self.pos[None]))
            tr.assert_close(k, m.turned(raw[1], "k_weight", self.pos[None]))
            ref = otr.attn(*(tr.f64(t) for t in (q, k, v)), self.h_parent, self.cu.cpu().numpy(), tr.f64(pk), tr.f64(pv),
                           self.cup.cpu().numpy(), m.d ** -0.5, softcap=self.softcap)
            assert_close(from_dev(out), None, ref, "verify", self.softcap)
        tl.assert_close(self.logits, olg.adjust(tr.f64(self.raw_logits), 1, own=self.paths, frequency=self.freq.cpu().numpy()), True)
        lp, ent, top, tlp = olp.token_logprobs(tr.f64(self.logits), self.tokens.cpu().numpy(), 4)
        assert np.abs(self.res["logprob"].cpu().numpy() - lp).max() < 1e-4
        assert np.abs(self.res["entropy"].cpu().numpy() - ent).max() < 1e-4
        assert np.array_equal(self.res["top_token"].cpu().numpy(), top)


@pytest.mark.parametrize("heads,softcap", [((16, 8, 128), 0.0), ((14, 2, 64), 30.0)], ids=str)
def test_verify_step(heads, softcap):
    import torch
    s = Verify(heads, softcap)
    want = {n: t.clone() for n, t in s.run().items()}
    s.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for t in s.res.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[n]) for n, t in s.res.items())
