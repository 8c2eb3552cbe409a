"""GPU: verify steps in a row, whose accepted tokens are appended to every request's cache where it lies.  The free rows
behind a request's prefix are the prefix of a request without nodes."""
import math

import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from attention_packed_varlen_causal_gb300 import workloads as wl
from oracle import tree as otr
from tests import test_gpu_tree as tt
from tests.helpers import from_dev, i32_dev, to_dev
from tests.test_gpu_shared import assert_close, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


class Caches:
    """Caches of `room` rows for each request, side by side; what is not taken yet is NaN."""

    def __init__(self, seed, lengths, nodes, room, heads):
        self.rng = np.random.default_rng(seed)
        self.lengths, self.nodes, self.room, self.heads = list(lengths), nodes, room, heads
        Hq, Hkv, d = heads
        R = len(lengths)
        self.k, self.v = (np.full((R * room, Hkv, d), 0x7FC0, np.uint16) for _ in range(2))
        for r, n in enumerate(lengths):
            self.k[r * room:r * room + n], self.v[r * room:r * room + n] = self.normal(n, Hkv), self.normal(n, Hkv)
        self.cu_nodes = np.concatenate(([0], *[[c, c] for c in np.cumsum(nodes)])).astype(np.int32)

    def normal(self, n, h):
        return wl.bf16_bits_from_f32(self.rng.standard_normal((n, h, self.heads[2]), dtype=np.float32))

    def cu_prefix(self):
        at = [(r * self.room + n, (r + 1) * self.room) for r, n in enumerate(self.lengths)]
        return np.concatenate(([0], *at)).astype(np.int32)

    def draft(self):
        Hq, Hkv, _ = self.heads
        T = sum(self.nodes)
        parent = np.array([p for n in self.nodes for p in tt.grow(self.rng, n, "random")], np.int32)
        return dict(q=self.normal(T, Hq), k=self.normal(T, Hkv), v=self.normal(T, Hkv), parent=parent)

    def reference(self, x, scale, softcap):
        """The same step on tightly packed prefixes."""
        keep = np.concatenate([np.arange(n) + r * self.room for r, n in enumerate(self.lengths)]).astype(np.int64)
        return otr.attn(f64(x["q"]), f64(x["k"]), f64(x["v"]), x["parent"], np.concatenate(([0], np.cumsum(self.nodes))),
                        f64(self.k[keep]), f64(self.v[keep]), np.concatenate(([0], np.cumsum(self.lengths))), scale, softcap=softcap)

    def accept(self, x):
        """Of each request the path to some node joins its cache; returns (node rows, cache rows)."""
        rows, places, a = [], [], 0
        for r, n in enumerate(self.nodes):
            if n:
                path = [a + i for i in otr.path(x["parent"][a:a + n], int(self.rng.integers(n)))]
                path = path[:self.room - self.lengths[r]]
                at = r * self.room + self.lengths[r] + np.arange(len(path))
                self.k[at], self.v[at] = x["k"][path], x["v"][path]
                self.lengths[r] += len(path)
                rows += path
                places += at.tolist()
            a += n
        return rows, places


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("lengths,nodes,room", [([300, 0, 121, 507], [26, 7, 40, 9], 520), ([3000, 40], [60, 60], 3300)], ids=["short", "long"])
@pytest.mark.parametrize("heads", [(16, 8, 128), (14, 2, 64)], ids=lambda h: "h%d_%d_d%d" % h)
def test_caches_that_grow_in_place(heads, lengths, nodes, room, softcap):
    """Four steps: the call on the caches as they lie equals the oracle on packed ones; one captured step, replayed on the
    next offsets and rows, gives the calls' bits."""
    import torch
    Hq, Hkv, d = heads
    c = Caches(1, lengths, nodes, room, heads)
    R, T, scale = len(lengths), sum(nodes), 1 / math.sqrt(d)
    pk, pv, cu, cup = to_dev(c.k), to_dev(c.v), i32_dev(c.cu_nodes), i32_dev(c.cu_prefix())
    ws = torch.empty(bg.bg_tree_attn_workspace_size(2 * R, T, max(nodes), room, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, graph = None, None
    for step in range(4):
        x = c.draft()
        new = {n: to_dev(x[n]) for n in ("q", "k", "v")}
        new["parent"] = i32_dev(x["parent"])
        if t is None:
            t, out = new, torch.empty_like(new["q"])
        for n in t:
            t[n].copy_(new[n])

        def run(o):
            bg.bg_tree_attn(t["q"], t["k"], t["v"], t["parent"], cu, max(nodes), pk, pv, cup, room, o, scale=scale,
                            softcap=softcap, workspace=ws, dev_status=st)
        want = torch.empty_like(out)
        run(want)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert_close(from_dev(want), None, c.reference(x, scale, softcap), f"step {step}", softcap)
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run(out)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        rows, places = (torch.tensor(i, device="cuda") for i in c.accept(x))
        pk[places], pv[places] = t["k"][rows], t["v"][rows]
        cup.copy_(i32_dev(c.cu_prefix()))
