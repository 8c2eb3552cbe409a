"""Edges of bg_token_logprobs on the GPU: waits that run out, and rows whose best logits lie in few places
(label sets, grammars, ties), in their results and in their time."""
import time

import numpy as np
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from tests.test_gpu_logprobs import check, logits, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


@pytest.mark.parametrize("N,V,stalled", [(3, 20001, 3), (1300, 5001, 700), (500, 20001, 0), (100, 30000, 60), (2, 60000, 1)],
                         ids=["none", "4_warps", "8_warps", "16_warps", "cluster"])
def test_rows_that_never_arrive(N, V, stalled):
    """The waits give up after a second; rows that were not computed say so, the others are right."""
    import torch
    x = logits(51, N, V, "float32").cuda()
    tok = np.arange(N) % V
    ref = run(x, tok, 1)
    out = {n: torch.full_like(t, 55) for n, t in ref.items()}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    bg.bg_selftest_logprobs_timeout(x, torch.as_tensor(tok.astype(np.int32)).cuda(), stalled, dev_status=st, **out)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 4
    assert int(st.item()) == (bg.BG_DEVSTAT_TIMEOUT if stalled < N else 0)
    for n in ref:
        assert torch.equal(out[n][:stalled], ref[n][:stalled]), n
        left = out[n][stalled:]
        assert (left == -1).all() if n == "top_token" else torch.isnan(left).all(), n
    check(x[:3, :4000], 5, "a call after it")


def restrict(x, low, seed):
    """Every row of x gets one of the patterns that leave few live logits, or most of them in few places."""
    import torch
    N, V = x.shape
    gen = torch.Generator().manual_seed(seed)
    lows = [-float("inf"), torch.finfo(x.dtype).min, -1e4] if low is None else [low]

    def some(n):
        return int(torch.randint(n, (1,), generator=gen))

    for i in range(N):
        live = torch.zeros(V, dtype=torch.bool)
        pattern, n = i % 8, [1, 2, 16, 37, 100, 700, 2500, 6000][(i // 8) % 8]
        n = min(n, V)
        at = some(V - n + 1)
        if pattern == 0:
            live[at:at + n] = True                       # neighbours: a label set
        elif pattern == 1:
            live[torch.randperm(V, generator=gen)[:n]] = True
        elif pattern == 2:
            live[V - n:] = True
            x[i, V - n:] = x[i, V - n:].sort().values    # rising to the row's end
        elif pattern == 3:
            live[some(64)::4096] = True                  # in one lane
        elif pattern == 4:
            live = (torch.arange(V) % 4096) < 256        # in one warp
            x[i, live] = x[i, live].sort().values
        elif pattern == 5:
            live[:] = True
            x[i, V - n:] = 40.0                          # equal ones at the end
        elif pattern == 6:
            live[at:at + n] = True
            x[i] = (x[i] * 0.5).round()                  # ... and equal ones among the live
        else:
            live[:] = True
        x[i, ~live] = lows[(i // 64 + i) % len(lows)]
    return x


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,V", [(128, 8003), (700, 9001), (500, 50001), (200, 20001), (70, 40001), (9, 130003)],
                         ids=["short", "4_warps", "8_warps", "16_warps", "2_ctas", "8_ctas"])
def test_few_live_logits(N, V, dtype):
    x = restrict(logits(52, N, V, dtype), None, 52)
    for K in (1, 5, 20, 32):
        check(x, K, f"{N} x {V} K {K}")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [300, 577, 600, 775, 831, 840, 1500, 2400])
def test_rows_about_as_long_as_the_list(V, dtype):
    for N in (1, 700):
        x = logits(53, N, V, dtype)
        for K in (25, 32):
            check(x, K, f"{N} x {V} K {K}")
    check(restrict(logits(54, 64, V, dtype), None, 54), 32, f"restricted {V}")


def test_rising_rows_of_many_sweeps():
    """All live logits in one warp's lanes and rising: the worst order for a list that keeps the first ones."""
    import torch
    x = torch.full((2, 1 << 20), -float("inf"))
    live = (torch.arange(1 << 20) % 4096) < 128
    x[0, live] = torch.linspace(-30, 30, int(live.sum()))
    x[1] = torch.linspace(-30, 30, 1 << 20)
    check(x, 32, "fp32")
    check(x.to(torch.bfloat16), 32, "bf16")


@pytest.mark.parametrize("low", [-float("inf"), -3e38], ids=["banned", "lowest"])
@pytest.mark.parametrize("N,V,dtype", [(480, 50001, "float32"), (200, 50001, "float32"), (2000, 65536, "bfloat16")])
def test_label_sets_take_about_the_time_of_other_rows(N, V, dtype, low):
    """Logits of all tokens but a few neighbours are banned: the row is read once, as any other (with a pass
    over it per alternative it took 7 to 160 times as long)."""
    import torch
    x = logits(55, 8, V, dtype).cuda().repeat(N // 8, 1)
    out = dict(top_token=torch.empty((N, 20), dtype=torch.int32, device="cuda"),
               top_logprob=torch.empty((N, 20), device="cuda"))

    def best_ms(y):
        ms = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(5):
                bg.bg_token_logprobs(y, **out)
            b.record()
            b.synchronize()
            ms.append(a.elapsed_time(b))
        return min(ms)

    ordinary = best_ms(x)
    for n in (1, 16, 100, 2000):
        y = torch.full_like(x, low)
        y[:, 12345:12345 + n] = x[:, :n]
        assert best_ms(y) < 3 * ordinary, n
