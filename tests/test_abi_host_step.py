"""Host-side refusals of the calls around a decode or verify step (norm and rotation, logit adjustments, tree
attention), which need no GPU: the C ABI rejects bad arguments before anything is enqueued, and the binding bad tensors."""
import ctypes
import math

import pytest
import torch

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build

INV, UNS, OK = bg.BG_ERR_INVALID_ARG, bg.BG_ERR_UNSUPPORTED, bg.BG_OK
F = 1 << 32            # fake pointers, 4 GB apart: never dereferenced, every call below ends on the host
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bg.load()


# ------------------------------------------------------------------ norm and rotation
ROPE = dict(q=F, qs=512, k=2 * F, ks=256, v=3 * F, vs=256, T=10, R=2, W=5, Hq=4, Hkv=2, d=128, qw=4 * F, kw=5 * F, eps=1e-6,
            off=0.0, pos=6 * F, axes=1, axis=None, step=3, f=7 * F, rot=128, inter=0, scale=1.0, qo=8 * F, ko=9 * F,
            vo=10 * F, smax=4, slot=3)


def packed(lib, **kw):
    a = {**ROPE, **kw}
    return lib.bg_packed_qk_norm_rope(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["Hq"], a["Hkv"], a["d"],
                                      a["qw"], a["kw"], a["eps"], a["off"], a["pos"], a["axes"], a["axis"], a["f"], a["rot"],
                                      a["inter"], a["scale"], a["qo"], a["ko"], a["vo"], None)


def beam(lib, **kw):
    a = {**ROPE, **kw}
    return lib.bg_beam_qk_norm_rope(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["R"], a["W"], a["Hq"], a["Hkv"],
                                    a["d"], a["qw"], a["kw"], a["eps"], a["off"], a["pos"], a["axes"], a["axis"], a["step"],
                                    a["f"], a["rot"], a["inter"], a["scale"], a["qo"], a["ko"], a["vo"], a["smax"],
                                    a["slot"], None)


def axis_array(*values):
    return (ctypes.c_int32 * 64)(*values)


BOTH = [
    (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(Hq=5), INV), (dict(d=0), INV), (dict(d=96), UNS), (dict(rot=0), INV),
    (dict(rot=24), UNS), (dict(rot=144), UNS), (dict(axes=0), INV), (dict(axes=5, axis=axis_array()), UNS),
    (dict(axes=2), INV), (dict(axes=2, axis=axis_array(0, 2)), INV), (dict(axes=2, axis=axis_array(0, -1)), INV),
    (dict(inter=2), INV), (dict(eps=-1.0), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV), (dict(off=INF), INV),
    (dict(scale=NAN), INV), (dict(qw=None), INV), (dict(kw=None), INV), (dict(qs=504), INV), (dict(ks=248), INV),
    (dict(vs=248), INV), (dict(qs=516), INV), (dict(ks=257), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(pos=None), INV), (dict(f=None), INV), (dict(qo=None), INV), (dict(ko=None), INV), (dict(q=F + 8), INV),
    (dict(v=3 * F + 2), INV), (dict(qo=8 * F + 8), INV), (dict(qw=4 * F + 8), INV), (dict(pos=6 * F + 2), INV),
    (dict(f=7 * F + 1), INV), (dict(qo=2 * F), INV), (dict(ko=F + 4096), INV), (dict(vo=9 * F), INV), (dict(ko=6 * F), INV),
    (dict(Hq=1 << 17, qs=1 << 24), UNS), (dict(qs=1 << 40), INV), (dict(vs=(1 << 31) + 8), INV),
    (dict(qo=F, qs=520), INV), (dict(qo=F + 1024), INV), (dict(vo=2 * F), INV), (dict(qo=4 * F - 512), INV)]


@pytest.mark.parametrize("call", [packed, beam], ids=["packed", "beam"])
@pytest.mark.parametrize("kw,expect", BOTH, ids=str)
def test_rope_refusals(lib, call, kw, expect):
    assert call(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [(dict(T=-1), INV), (dict(v=None), INV), (dict(vo=None), INV),
                                       (dict(T=0, q=None, k=None, v=None, vo=None, pos=None), OK)], ids=str)
def test_packed_rope_refusals(lib, kw, expect):
    assert packed(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(R=-1), INV), (dict(W=0), INV), (dict(smax=0), INV), (dict(slot=-1), INV), (dict(slot=4), INV), (dict(step=-1), INV),
    (dict(smax=17), UNS), (dict(v=None), INV), (dict(vo=None), INV), (dict(v=None, vo=None), INV),
    # a slot that is not written counts as well: the suffix is one buffer
    (dict(ko=9 * F, vo=9 * F + 10 * 4 * 512 - 512), INV), (dict(k=9 * F + 512, ks=1024), INV),
    (dict(R=0), OK), (dict(R=0, q=None, k=None, v=None, ko=None, vo=None), OK)], ids=str)
def test_beam_rope_refusals(lib, kw, expect):
    assert beam(lib, **kw) == expect


# ------------------------------------------------------------------ logits
LOG = dict(x=F, idt=0, istr=100, G=3, per=2, V=100, pt=2 * F, cup=3 * F, P=20, own=4 * F, lens=5 * F, S=6, rep=6 * F,
           freq=7 * F, pres=8 * F, bt=9 * F, bv=10 * F, cub=11 * F, B=7, mask=12 * F, ms=4, M=5, mi=13 * F, out=14 * F, odt=0,
           ostr=100, st=None)


def adjust(lib, **kw):
    a = {**LOG, **kw}
    return lib.bg_adjust_logits(a["x"], a["idt"], a["istr"], a["G"], a["per"], a["V"], a["pt"], a["cup"], a["P"], a["own"],
                                a["lens"], a["S"], a["rep"], a["freq"], a["pres"], a["bt"], a["bv"], a["cub"], a["B"],
                                a["mask"], a["ms"], a["M"], a["mi"], a["out"], a["odt"], a["ostr"], a["st"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(G=-1), INV), (dict(per=0), INV), (dict(P=-1), INV), (dict(S=-1), INV), (dict(B=-1), INV), (dict(M=-1), INV),
    (dict(idt=2), INV), (dict(odt=-1), INV), (dict(V=0), UNS), (dict(V=bg.BG_MAX_VOCAB + 1, istr=1 << 23, ostr=1 << 23), UNS),
    (dict(S=bg.BG_MAX_SEQLEN + 1), UNS), (dict(odt=1), UNS), (dict(istr=99), INV), (dict(ostr=99), INV), (dict(ms=3), INV), (dict(istr=1 << 50), INV),
    (dict(ostr=1 << 32), INV), (dict(ms=1 << 62), INV),
    (dict(mask=None), INV), (dict(mask=None, mi=None), INV), (dict(mi=None), INV), (dict(G=1 << 20, per=1 << 12), UNS), (dict(G=1, per=(1 << 30) + 1), UNS),
    (dict(x=None), INV), (dict(out=None), INV), (dict(pt=None), INV), (dict(cup=None), INV), (dict(own=None), INV),
    (dict(bt=None), INV), (dict(bv=None), INV), (dict(cub=None), INV), (dict(x=F + 2), INV), (dict(out=14 * F + 2), INV),
    (dict(x=F + 1, idt=1), INV), (dict(pt=2 * F + 2), INV), (dict(lens=5 * F + 1), INV), (dict(mask=12 * F + 2), INV),
    (dict(st=15 * F + 2), INV), (dict(rep=6 * F + 3), INV), (dict(out=F + 400), INV), (dict(out=F, ostr=104), INV),
    (dict(out=F, idt=1), INV), (dict(out=2 * F - 1200), INV), (dict(out=13 * F), INV), (dict(out=8 * F - 4), INV),
    (dict(st=14 * F + 8), INV), (dict(G=0), OK), (dict(G=0, x=None, out=None, mask=None, M=0, mi=None), OK)], ids=str)
def test_adjust_refusals(lib, kw, expect):
    assert adjust(lib, **kw) == expect


# ------------------------------------------------------------------ trees
TREE = dict(q=F, k=2 * F, v=3 * F, par=4 * F, cu=5 * F, R=3, T=10, maxn=8, pk=6 * F, pv=7 * F, cup=8 * F, P=12, maxp=9, Hq=4,
            Hkv=2, d=64, scale=0.125, cap=0.0, out=9 * F, lse=None, ws=10 * F, wsb=1 << 30, st=None)


def tree(lib, name, **kw):
    a = {**TREE, **kw}
    if name == "bg_tree_plan":
        return lib.bg_tree_plan(a["par"], a["cu"], a["R"], a["T"], a["maxn"], a["cup"], a["P"], a["maxp"], a["Hq"], a["Hkv"],
                                a["d"], a["ws"], a["wsb"], a["st"], None)
    return getattr(lib, name)(a["q"], a["k"], a["v"], a["par"], a["cu"], a["R"], a["T"], a["maxn"], a["pk"], a["pv"],
                              a["cup"], a["P"], a["maxp"], a["Hq"], a["Hkv"], a["d"], a["scale"], a["cap"], a["out"],
                              a["lse"], a["ws"], a["wsb"], a["st"], None)


PLANS = [
    (dict(R=-1), INV), (dict(T=-1), INV), (dict(P=-1), INV), (dict(maxn=-1), INV), (dict(maxp=-1), INV), (dict(R=0), INV),
    (dict(Hq=5), INV), (dict(Hkv=0), INV), (dict(d=96), UNS), (dict(Hq=258), UNS), (dict(maxn=bg.BG_MAX_TREE + 1), UNS),
    (dict(maxp=bg.BG_MAX_SEQLEN + 1), UNS), (dict(par=None), INV), (dict(cu=None), INV), (dict(cup=None), INV),
    (dict(par=4 * F + 2), INV), (dict(cu=5 * F + 1), INV), (dict(ws=None), INV), (dict(ws=10 * F + 128), INV),
    (dict(wsb=100), INV), (dict(ws=4 * F), INV), (dict(par=10 * F + 512), INV), (dict(st=10 * F + 4), INV),
    (dict(st=11 * F + 2), INV)]
RUNS = [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(out=None), INV), (dict(pk=None), INV),
    (dict(q=F + 8), INV), (dict(scale=0.0), INV), (dict(scale=NAN), INV), (dict(scale=3e38), INV), (dict(cap=-1.0), INV),
    (dict(cap=INF), INV), (dict(out=F), INV), (dict(out=4 * F), INV), (dict(out=10 * F), INV), (dict(lse=9 * F + 64), INV),
    (dict(lse=4 * F + 4), INV), (dict(st=9 * F), INV)]


@pytest.mark.parametrize("name", ["bg_tree_attn", "bg_tree_attn_planned"])
@pytest.mark.parametrize("kw,expect", PLANS + RUNS, ids=str)
def test_tree_refusals(lib, name, kw, expect):
    assert tree(lib, name, **kw) == expect


@pytest.mark.parametrize("kw,expect", PLANS, ids=str)
def test_tree_plan_refusals(lib, kw, expect):
    assert tree(lib, "bg_tree_plan", **kw) == expect


def test_no_nodes_is_a_noop(lib):
    none = dict(q=None, k=None, v=None, par=None, cu=None, cup=None, out=None, ws=None, T=0)
    assert tree(lib, "bg_tree_attn", **none) == OK and tree(lib, "bg_tree_plan", **none) == OK
    assert tree(lib, "bg_tree_attn", R=0, P=0, **none) == OK


def test_tree_workspace_size():
    size = bg.bg_tree_attn_workspace_size
    assert size(32, 2000, 64, 500, 16, 8, 128) % 256 == 0
    # whole key tiles of bits for each node
    assert size(1, 1000, 1000, 100, 4, 2, 64) - size(1, 1000, 100, 100, 4, 2, 64) >= 1000 * 7 * 16
    for bad in ((-1, 5, 5, 5, 4, 2, 64), (1, 5, 5, 5, 5, 2, 64), (1, 5, 5, 5, 4, 2, 80), (1, 5, 1025, 5, 4, 2, 64),
                (0, 5, 5, 5, 4, 2, 64), (1, 1 << 33, 5, 5, 4, 2, 64)):
        assert size(*bad) == 0


# ------------------------------------------------------------------ the binding
def test_binding_refuses_wrong_tensors(lib):
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    z = torch.zeros

    def rope(**kw):
        t = dict(q=z(10, 4, 128, dtype=bf), k=z(10, 2, 128, dtype=bf), v=z(10, 2, 128, dtype=bf), positions=z(10, dtype=i32),
                 q_out=z(10, 4, 128, dtype=bf), k_out=z(10, 2, 128, dtype=bf), v_out=z(10, 2, 128, dtype=bf), inv_freq=z(64))
        t.update(kw)
        bg.bg_packed_qk_norm_rope(**t)

    for bad in (dict(q=z(10, 4, 128)), dict(k=z(9, 2, 128, dtype=bf)), dict(v=z(10, 2, 64, dtype=bf)),
                dict(q=z(10, 128, 4, dtype=bf).transpose(1, 2)), dict(q=z(10, 4, 256, dtype=bf)[..., ::2]),
                dict(q=z(10, 8, 128, dtype=bf)[:, ::2]), dict(positions=z(9, dtype=i32)), dict(positions=z(10)),
                dict(positions=z(1, 1, 10, dtype=i32)), dict(positions=z(10, 2, dtype=i32).T), dict(inv_freq=z(64).double()),
                dict(inv_freq=z(8, 8)), dict(q_weight=z(64, dtype=bf), k_weight=z(64, dtype=bf)),
                dict(q_out=z(10, 4, 64, dtype=bf)), dict(k_out=z(10, 4, 128, dtype=bf)[:, ::2]), dict(v_out=z(10, 2, 128)),
                dict(axis_of=[0] * 63), dict(q_out=z(10, 4, 128, dtype=bf, device="meta")), {}):
        with pytest.raises(ValueError):
            rope(**bad)                       # the last one: everything right, but not on a CUDA device

    def beams(**kw):
        t = dict(q=z(2, 5, 4, 128, dtype=bf), k=z(2, 5, 2, 128, dtype=bf), v=z(2, 5, 2, 128, dtype=bf), base_pos=z(2, dtype=i32),
                 step=1, q_out=z(2, 5, 4, 128, dtype=bf), suffix_k=z(2, 5, 4, 2, 128, dtype=bf),
                 suffix_v=z(2, 5, 4, 2, 128, dtype=bf), slot=0, inv_freq=z(64))
        t.update(kw)
        bg.bg_beam_qk_norm_rope(**t)

    for bad in (dict(q=z(2, 6, 4, 128, dtype=bf)[:, :5]), dict(base_pos=z(5, dtype=i32)), dict(base_pos=z(3, 3, dtype=i32)),
                dict(suffix_v=z(2, 5, 3, 2, 128, dtype=bf)), dict(suffix_k=z(2, 5, 4, 4, 128, dtype=bf)[:, :, :, ::2]),
                dict(k=z(2, 5, 2, 128)), dict(q_out=z(10, 4, 128, dtype=bf)), {}):
        with pytest.raises(ValueError):
            beams(**bad)

    def logits(**kw):
        t = dict(logits=z(6, 100), out=z(6, 100), rows_per_group=2, prompt_tokens=z(20, dtype=i32), cu_prompt=z(4, dtype=i32),
                 own_tokens=z(6, 5, dtype=i32), own_lens=z(6, dtype=i32), repetition=z(3), frequency=z(3), presence=z(3),
                 bias_tokens=z(7, dtype=i32), bias_values=z(7), cu_bias=z(4, dtype=i32), mask=z(5, 4, dtype=i32),
                 mask_index=z(6, dtype=i32))
        t.update(kw)
        bg.bg_adjust_logits(**t)

    for bad in (dict(logits=z(6, 100, dtype=torch.float16)), dict(out=z(6, 101)), dict(out=z(100, 6).T), dict(rows_per_group=4),
                dict(rows_per_group=0), dict(cu_prompt=z(3, dtype=i32)), dict(cu_prompt=None), dict(prompt_tokens=None),
                dict(prompt_tokens=z(20, dtype=torch.int64)), dict(own_tokens=z(5, 5, dtype=i32)), dict(own_tokens=z(6, dtype=i32)),
                dict(own_lens=z(5, dtype=i32)), dict(repetition=z(6)), dict(frequency=z(3).double()), dict(bias_values=None),
                dict(bias_values=z(6)), dict(cu_bias=z(3, dtype=i32)), dict(mask=z(5, 4)), dict(mask=z(20, dtype=i32)),
                dict(mask_index=z(3, dtype=i32)), dict(out=z(6, 100, device="meta")), {}):
        with pytest.raises(ValueError):
            logits(**bad)

    def nodes(**kw):
        t = dict(q=z(10, 4, 64, dtype=bf), k=z(10, 2, 64, dtype=bf), v=z(10, 2, 64, dtype=bf), parent=z(10, dtype=i32),
                 cu_nodes=z(4, dtype=i32), max_nodes=8, prefix_k=z(12, 2, 64, dtype=bf), prefix_v=z(12, 2, 64, dtype=bf),
                 cu_prefix=z(4, dtype=i32), max_prefix_len=9, out=z(10, 4, 64, dtype=bf),
                 workspace=z(1 << 20, dtype=torch.uint8))
        t.update(kw)
        bg.bg_tree_attn(**t)

    for bad in (dict(q=z(10, 4, 64)), dict(parent=z(9, dtype=i32)), dict(parent=z(10, dtype=torch.int64)), dict(prefix_v=None),
                dict(cu_prefix=z(3, dtype=i32)), dict(out=z(10, 4, 128, dtype=bf)[..., ::2]), dict(lse=z(4, 10)),
                dict(workspace=None), dict(v=z(10, 2, 32, dtype=bf)), {}):
        with pytest.raises(ValueError):
            nodes(**bad)


def test_sizes_that_do_not_fit_are_refused(lib, monkeypatch):
    """A size past int32 would reach the C ABI as its low 32 bits."""
    monkeypatch.setattr(bg, "_launch", lambda *a: pytest.fail("launched"))
    meta = dict(device="meta")
    x = torch.empty((1, 1 << 33), **meta)
    with pytest.raises(bg.BgError):
        bg.bg_adjust_logits(x, x)
    with pytest.raises(bg.BgError):
        bg.bg_beam_qk_norm_rope(*(torch.empty((2, 5, h, 64), dtype=torch.bfloat16, **meta) for h in (2, 2, 2)),
                                torch.empty(2, dtype=torch.int32, **meta), 1 << 32,
                                torch.empty((2, 5, 2, 64), dtype=torch.bfloat16, **meta),
                                *(torch.empty((2, 5, 1, 2, 64), dtype=torch.bfloat16, **meta) for _ in range(2)), 0,
                                inv_freq=torch.empty(32, **meta))
