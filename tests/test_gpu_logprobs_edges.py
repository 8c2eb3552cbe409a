"""Edges of bg_token_logprobs on the GPU: waits that run out."""
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
