"""Host-side refusals of the shared-prefix attention and log-probability calls, which need no GPU:
the C ABI rejects bad arguments before anything is enqueued, and the binding bad tensors."""
import math

import pytest
import torch

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build

INV, UNS, OK = bg.BG_ERR_INVALID_ARG, bg.BG_ERR_UNSUPPORTED, bg.BG_OK
F = 1 << 32            # fake pointers, 4 GB apart: never dereferenced, every call below ends on the host


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bg.load()


BASE = dict(q=F, k=2 * F, v=3 * F, cu=4 * F, S=3, T=10, maxlen=8, pk=5 * F, pv=6 * F, cup=7 * F, P=12, maxp=9, cug=8 * F,
            R=2, Hq=4, Hkv=2, d=64, scale=0.125, cap=0.0, out=9 * F, lse=None, ws=10 * F, wsb=1 << 30, st=None)


def run(lib, name, **kw):
    a = {**BASE, **kw}
    return getattr(lib, name)(a["q"], a["k"], a["v"], a["cu"], a["S"], a["T"], a["maxlen"], a["pk"], a["pv"], a["cup"],
                              a["P"], a["maxp"], a["cug"], a["R"], a["Hq"], a["Hkv"], a["d"], a["scale"], a["cap"],
                              a["out"], a["lse"], a["ws"], a["wsb"], a["st"], None)


def plan(lib, name, **kw):
    a = {**BASE, **kw}
    return getattr(lib, name)(a["cu"], a["S"], a["T"], a["maxlen"], a["cup"], a["P"], a["maxp"], a["cug"], a["R"],
                              a["Hq"], a["Hkv"], a["d"], a["ws"], a["wsb"], a["st"], None)


SIZES = [
    (dict(S=-1), INV), (dict(T=-1), INV), (dict(R=-1), INV), (dict(P=-1), INV), (dict(maxlen=-1), INV),
    (dict(maxp=-1), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(d=0), INV), (dict(Hq=5), INV),
    (dict(R=0), INV), (dict(R=0, S=0), INV), (dict(d=96), UNS), (dict(Hq=258), UNS),
    (dict(maxlen=bg.BG_MAX_SEQLEN + 1), UNS), (dict(maxp=bg.BG_MAX_SEQLEN + 1), UNS),
    (dict(cu=None), INV), (dict(cup=None), INV), (dict(cug=None), INV), (dict(cu=4 * F + 2), INV),
    (dict(ws=None), INV), (dict(ws=10 * F + 128), INV), (dict(wsb=255), INV), (dict(st=F + 2), INV),
    (dict(ws=4 * F), INV), (dict(ws=7 * F), INV), (dict(ws=8 * F), INV),
    (dict(R=0, S=0, T=0, P=0), OK),
]
RUNS = [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(pk=None), INV), (dict(pv=None), INV),
    (dict(out=None), INV), (dict(q=F + 8), INV), (dict(k=F + 8), INV), (dict(pv=F + 8), INV), (dict(out=F + 8), INV),
    (dict(lse=F + 2), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.nan), INV),
    (dict(scale=math.inf), INV), (dict(cap=-1.0), INV), (dict(cap=math.nan), INV), (dict(cap=math.inf), INV),
    (dict(cap=1e-39), INV), (dict(cap=3e38), INV), (dict(scale=1e30, cap=1e-20), INV),
    (dict(out=F), INV), (dict(out=2 * F), INV), (dict(out=3 * F + 256), INV), (dict(out=5 * F), INV),
    (dict(out=6 * F), INV), (dict(out=7 * F), INV), (dict(lse=F), INV), (dict(lse=9 * F), INV), (dict(lse=10 * F), INV),
    (dict(ws=F), INV), (dict(ws=9 * F), INV), (dict(ws=5 * F), INV),
]


@pytest.mark.parametrize("name", ["bg_shared_prefill_attn", "bg_shared_prefill_attn_planned",
                                  "bg_shared_last_token_attn", "bg_shared_last_token_attn_planned"])
@pytest.mark.parametrize("kw,expect", SIZES + RUNS, ids=str)
def test_run_refusals(lib, name, kw, expect):
    assert run(lib, name, **kw) == expect


@pytest.mark.parametrize("name", ["bg_shared_prefill_plan", "bg_shared_last_token_plan"])
@pytest.mark.parametrize("kw,expect", SIZES, ids=str)
def test_plan_refusals(lib, name, kw, expect):
    assert plan(lib, name, **kw) == expect


def test_no_queries_is_a_noop(lib):
    """Before any pointer is looked at: no tokens (prefill), no samples (both)."""
    none = dict(q=None, k=None, v=None, cu=None, cup=None, cug=None, out=None, ws=None)
    assert run(lib, "bg_shared_prefill_attn", T=0, **none) == OK
    assert run(lib, "bg_shared_last_token_attn", S=0, T=0, **none) == OK
    assert run(lib, "bg_shared_last_token_attn", S=3, T=0, **none) == INV      # three queries over the prefixes


def test_workspace_size():
    size = bg.bg_shared_attn_workspace_size
    assert size(32, 480, 27000, 96, 500, 16, 8, 128) % 256 == 0
    # key ranges of a few tiles are never split, longer ones bring room for partial results
    assert size(1, 4, 40, 20, 100, 16, 8, 128) < 50_000 < 1_000_000 < size(1, 4, 40, 20, 4096, 16, 8, 128)
    assert size(4, 128, 26000, 400, 32768, 32, 8, 128) < 64 << 20
    for bad in ((-1, 5, 5, 5, 5, 4, 2, 64), (1, 5, 5, 5, 5, 5, 2, 64), (1, 5, 5, 5, 5, 4, 2, 80),
                (1, 5, 5, 70000, 5, 4, 2, 64), (0, 5, 5, 5, 5, 4, 2, 64)):
        assert size(*bad) == 0


LP = dict(x=F, dtype=bg.BG_DTYPE_F32, stride=100, N=4, V=100, tok=2 * F, K=3, lp=3 * F, ent=4 * F, tt=5 * F, tl=6 * F,
          st=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), INV), (dict(dtype=2), INV), (dict(dtype=-1), INV), (dict(V=0), UNS), (dict(K=-1), UNS),
    (dict(K=33), UNS), (dict(V=2, stride=2, K=3), UNS), (dict(V=bg.BG_MAX_VOCAB + 1, stride=1 << 23), UNS),
    (dict(stride=99), INV), (dict(x=None), INV), (dict(x=F + 2), INV), (dict(x=F + 1, dtype=1), INV),
    (dict(tok=None), INV), (dict(lp=None), INV), (dict(tt=None), INV), (dict(tl=None), INV), (dict(K=0), INV),
    (dict(tok=2 * F + 1), INV), (dict(lp=3 * F + 1), INV), (dict(ent=F + 2), INV), (dict(st=F + 1), INV),
    (dict(tok=None, lp=None, ent=None, K=0, tt=None, tl=None), INV), (dict(lp=F), INV), (dict(ent=F + 1596), INV),
    (dict(tt=2 * F), INV), (dict(lp=4 * F), INV), (dict(tl=5 * F + 44), INV), (dict(N=0), OK),
    (dict(N=0, x=None, tok=None), OK)], ids=str)
def test_logprobs_refusals(lib, kw, expect):
    a = {**LP, **kw}
    assert lib.bg_token_logprobs(a["x"], a["dtype"], a["stride"], a["N"], a["V"], a["tok"], a["K"], a["lp"], a["ent"],
                                 a["tt"], a["tl"], a["st"], None) == expect


def test_binding_refuses_wrong_tensors(lib):
    """Types, shapes, layouts and devices are looked at before a pointer leaves Python."""
    bf, i32 = torch.bfloat16, torch.int32

    def shared(**kw):
        t = dict(q=torch.zeros(10, 4, 64, dtype=bf), k=torch.zeros(10, 2, 64, dtype=bf),
                 v=torch.zeros(10, 2, 64, dtype=bf), cu=torch.zeros(4, dtype=i32), pk=torch.zeros(12, 2, 64, dtype=bf),
                 pv=torch.zeros(12, 2, 64, dtype=bf), cup=torch.zeros(3, dtype=i32), cug=torch.zeros(3, dtype=i32),
                 out=torch.zeros(10, 4, 64, dtype=bf), lse=None, ws=torch.zeros(1 << 20, dtype=torch.uint8))
        t.update(kw)
        bg.bg_shared_prefill_attn(t["q"], t["k"], t["v"], t["cu"], 8, t["pk"], t["pv"], t["cup"], 9, t["cug"], t["out"],
                                  lse=t["lse"], workspace=t["ws"])

    for bad in (dict(q=torch.zeros(10, 4, 64)), dict(k=torch.zeros(10, 64, 2, dtype=bf).transpose(1, 2)),
                dict(v=torch.zeros(9, 2, 64, dtype=bf)), dict(cu=torch.zeros(4, dtype=torch.int64)),
                dict(pv=None), dict(pv=torch.zeros(12, 2, 32, dtype=bf)), dict(cup=torch.zeros(4, dtype=i32)),
                dict(out=torch.zeros(10, 4, 128, dtype=bf)[..., ::2]), dict(lse=torch.zeros(4, 10)), dict(ws=None),
                dict(out=torch.zeros(10, 4, 64, dtype=bf, device="meta")), {}):
        with pytest.raises(ValueError):
            shared(**bad)                       # the last one: everything right, but not on a CUDA device

    x = torch.zeros(4, 100)
    for bad in (dict(logits=x.double()), dict(logits=x.t()), dict(tokens=torch.zeros(4, dtype=torch.int64)),
                dict(entropy=torch.zeros(5)), dict(top_token=torch.zeros(4, 3, dtype=i32), top_logprob=torch.zeros(4, 2)),
                dict(top_token=torch.zeros(4, 3), top_logprob=torch.zeros(4, 3)), dict(entropy=torch.zeros(4))):
        with pytest.raises(ValueError):
            bg.bg_token_logprobs(**{"logits": x, **bad})
