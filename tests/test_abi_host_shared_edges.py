"""Host-side refusals of sizes that contradict each other or do not fit the C ABI's integers, in the
shared-prefix attention and log-probability calls (no GPU)."""
import types

import pytest
import torch

from attention_packed_varlen_causal_gb300 import binding as bg
from tests.test_abi_host_shared import F, INV, OK, UNS, lib, plan, run  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("kw", [dict(S=0), dict(S=0, P=0), dict(S=0, R=0, P=0)], ids=str)
def test_tokens_without_samples(lib, kw):  # noqa: F811
    """No sample holds the tokens: no query row would be written."""
    for name in ("bg_shared_prefill_attn", "bg_shared_prefill_attn_planned"):
        assert run(lib, name, **kw) == INV
    assert plan(lib, "bg_shared_prefill_plan", **kw) == INV
    # the last-token calls have a query per sample, so none here
    assert run(lib, "bg_shared_last_token_attn", **kw) == OK
    assert bg.bg_shared_attn_workspace_size(kw.get("R", 2), 0, 10, 8, 9, 4, 2, 64) == 0


def test_sizes_past_32_bits_are_refused_not_cut(lib):  # noqa: F811
    """The C ABI takes int32 sizes: 2^32 + 10 must not reach it as 10."""
    big, bf, i32 = (1 << 32) + 10, torch.bfloat16, torch.int32
    cu, cug = torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    q, k = torch.zeros(10, 4, 64, dtype=bf), torch.zeros(10, 2, 64, dtype=bf)
    for n, p in ((big, 9), (8, big), (-big, 9)):
        with pytest.raises(bg.BgError) as e:
            bg.bg_shared_prefill_attn(q, k, k, cu, n, k, k, cug, p, cug, q.clone(), workspace=ws)
        assert e.value.status == bg.BG_ERR_UNSUPPORTED
    for sizes in ((big, 8, 12, 9), (10, big, 12, 9), (10, 8, big, 9), (10, 8, 12, big)):
        T, n, P, p = sizes
        with pytest.raises(bg.BgError) as e:
            bg.bg_shared_last_token_plan(cu, T, n, cug, P, p, cug, 4, 2, 64, workspace=ws)
        assert e.value.status == bg.BG_ERR_UNSUPPORTED
        assert bg.bg_shared_attn_workspace_size(2, 3, T, n, p, 4, 2, 64) == 0 or P == big
    for shape in ((1, big), (big, 1)):
        with pytest.raises(bg.BgError) as e:
            bg.bg_token_logprobs(torch.empty(shape, dtype=bf, device="meta"), entropy=torch.zeros(1))
        assert e.value.status == bg.BG_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,expect", [
    (dict(N=0), INV), (dict(V=0), INV), (dict(row=-1), INV), (dict(row=5), INV), (dict(V=bg.BG_MAX_VOCAB + 1), UNS)] +
    [(dict([(n, p)]), INV) for n in ("x", "tok", "lp", "ent", "tt", "tl", "st") for p in (None, F + 2)], ids=str)
def test_logprobs_selftest_refusals(lib, kw, expect):  # noqa: F811
    a = {**dict(x=F, N=4, V=100, tok=2 * F, row=2, lp=3 * F, ent=4 * F, tt=5 * F, tl=6 * F, st=7 * F), **kw}
    assert lib.bg_selftest_logprobs_timeout(a["x"], a["N"], a["V"], a["tok"], a["row"], a["lp"], a["ent"], a["tt"],
                                            a["tl"], a["st"], None) == expect


def test_current_stream_without_torchs_shortcut(monkeypatch):
    """The current stream is found by the public call where torch has no private one."""
    seen = []
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: seen.append(i) or types.SimpleNamespace(cuda_stream=77))
    assert bg._raw_stream(3) == 77 and seen == [3]


def test_status_word_in_another_argument(lib):  # noqa: F811
    """dev_status is an argument too: outputs and the workspace do not overlap it."""
    for name in ("bg_shared_prefill_attn", "bg_shared_last_token_attn_planned"):
        for kw in (dict(st=9 * F + 4), dict(st=10 * F + 512), dict(lse=11 * F, st=11 * F + 8)):
            assert run(lib, name, **kw) == INV
    assert plan(lib, "bg_shared_prefill_plan", st=10 * F + 512) == INV
    lp = dict(x=F, N=4, V=100, tok=2 * F, K=3, lp=3 * F, ent=4 * F, tt=5 * F, tl=6 * F)
    for st in (3 * F + 4, 4 * F + 12, 5 * F + 44, 6 * F):
        assert lib.bg_token_logprobs(lp["x"], 0, 100, lp["N"], lp["V"], lp["tok"], lp["K"], lp["lp"], lp["ent"], lp["tt"],
                                     lp["tl"], st, None) == INV


def test_scale_past_the_range_of_base_two(lib):  # noqa: F811
    """The kernels take scores in base 2: 3e38 log2(e) is infinite."""
    for name in ("bg_shared_prefill_attn", "bg_shared_last_token_attn_planned"):
        assert run(lib, name, scale=3e38) == INV
