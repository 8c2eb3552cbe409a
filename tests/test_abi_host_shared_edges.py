"""Host-side refusals of sizes that contradict each other or do not fit the C ABI's integers, in the
shared-prefix attention and log-probability calls (no GPU)."""
import pytest

from attention_packed_varlen_causal_gb300 import binding as bg
from tests.test_abi_host_shared import INV, OK, lib, plan, run  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("kw", [dict(S=0), dict(S=0, P=0), dict(S=0, R=0, P=0)], ids=str)
def test_tokens_without_samples(lib, kw):  # noqa: F811
    """No sample holds the tokens: no query row would be written."""
    for name in ("bg_shared_prefill_attn", "bg_shared_prefill_attn_planned"):
        assert run(lib, name, **kw) == INV
    assert plan(lib, "bg_shared_prefill_plan", **kw) == INV
    # the last-token calls have a query per sample, so none here
    assert run(lib, "bg_shared_last_token_attn", **kw) == OK
    assert bg.bg_shared_attn_workspace_size(kw.get("R", 2), 0, 10, 8, 9, 4, 2, 64) == 0
