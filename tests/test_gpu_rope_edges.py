"""GPU edges of bg_packed_qk_norm_rope and bg_beam_qk_norm_rope: single rows in place."""
import pytest

from tests import test_gpu_rope as tr

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


@pytest.mark.parametrize("slots,slot", [(1, 0), (4, 0), (4, 2), (16, 15)])
@pytest.mark.parametrize("heads", [(6, 2, 128), (14, 2, 64), (1, 1, 64)], ids=lambda h: "h%d_%d_d%d" % h)
def test_one_beam_in_place(heads, slots, slot):
    """A search of one beam whose K and V already lie in their slot: the same bits as from rows of their own, and the
    other slots stay."""
    import torch
    Hq, Hkv, d = heads
    x = tr.inputs(31, 1, *heads)
    base = torch.tensor([77], dtype=torch.int32, device="cuda")
    q, k, v = (t.unflatten(0, (1, 1)) for t in tr.split(x))
    want_k, want_v = (torch.randn((1, 1, slots, Hkv, d), device="cuda").bfloat16() for _ in range(2))
    got_k, got_v = want_k.clone(), want_v.clone()
    want, got = torch.empty((1, 1, Hq, d), dtype=torch.bfloat16, device="cuda"), q.clone()
    bg.bg_beam_qk_norm_rope(q, k, v, base, 2, want, want_k, want_v, slot, **x["kw"])
    got_k[:, :, slot], got_v[:, :, slot] = k, v
    bg.bg_beam_qk_norm_rope(got, got_k[:, :, slot], got_v[:, :, slot], base, 2, got, got_k, got_v, slot, **x["kw"])
    assert all(torch.equal(a, b) for a, b in ((got, want), (got_k, want_k), (got_v, want_v)))
    # Q may stand alone in place, and only its own input may
    got = q.clone()
    bg.bg_beam_qk_norm_rope(got, k, v, base, 2, got, got_k, got_v, slot, **x["kw"])
    assert torch.equal(got, want)
    if slots > 1:
        other = got_k[:, :, (slot + 1) % slots]
        with pytest.raises(bg.BgError):
            bg.bg_beam_qk_norm_rope(q, other, v, base, 2, got, got_k, got_v, slot, **x["kw"])


def test_one_token_in_place_within_a_wider_row():
    import torch
    x = tr.inputs(32, 1, 6, 2, 128)
    want = tr.run(x)
    q, k, v = tr.split(x)                         # views of one row of the projection
    bg.bg_packed_qk_norm_rope(q, k, v, x["positions"], q, k, v, **x["kw"])
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), want))
