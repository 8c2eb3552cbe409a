"""GPU edges of bg_packed_qk_norm_rope and bg_beam_qk_norm_rope: single rows in place, and angles to the stated bound."""
import numpy as np
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


TWO_PI = 6283185307179586476925286766559005768394       # 10^39 times 2 pi


def turned_back(pos, freq):
    """pos * freq modulo 2 pi in (-pi, pi], exact to 2^-90: a product of whole numbers."""
    mant, exp = np.frexp(np.float64(freq))
    m, e = int(mant * (1 << 24)), 24 - int(exp)           # freq = m / 2^e
    turn = (TWO_PI << 128) // 10 ** 39
    r = ((int(pos) * m) << (128 - e)) % turn
    return float(r - turn if 2 * r > turn else r) / 2.0 ** 128


def places_near_zero(limit, half, seed):
    """Positions up to limit (past 2^24 where it is larger), frequencies, and the (row, frequency) places whose sine or cosine
    is below about 2^-11, with their exact angles."""
    rng = np.random.default_rng(seed)
    freq = np.concatenate((rng.uniform(0.75, 1.0, half // 2), 1e4 ** (-np.arange(half - half // 2) / half))).astype(np.float32)
    pos = rng.integers(max(-limit, -(1 << 31)), min(limit, (1 << 31) - 1), 400000, endpoint=True)
    if limit > 1 << 24:
        pos = pos[np.abs(pos) > 1 << 24]
    near = np.remainder(pos[:, None].astype(np.float64) * freq.astype(np.float64), np.pi / 2)      # good to 2^-20
    near = np.minimum(near, np.pi / 2 - near) < 2.0 ** -11
    keep = np.flatnonzero(near.any(1))[:40000]
    rows, cols = np.nonzero(near[keep])
    pos = pos[keep]
    return pos, freq, rows, cols, np.array([turned_back(pos[r], freq[c]) for r, c in zip(rows, cols)])


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("limit,off", [(1 << 16, 2.0 ** -19), (1 << 24, 2.0 ** -19), (1 << 31, 2.0 ** -17)], ids=["2^16", "2^24", "2^31"])
def test_angles_to_the_stated_bound(limit, off, d, interleaved):
    """Pairs (1, 0) without a norm become (cos, sin), each rounded to bf16 once.  Looked at where one of them is next to 0, so
    that its rounding (2^-8 of it) does not hide the angle's error: 2^-19 or 2^-17, and 2^-21 for the fast sine and cosine."""
    import torch
    half = d // 2
    pos, freq, rows, cols, angle = places_near_zero(limit, half, d)
    assert len(rows) > 7000
    x = torch.zeros((len(pos), 2, half), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    x = (x.transpose(1, 2) if interleaved else x).reshape(len(pos), 1, d).contiguous()
    q, k = torch.empty_like(x), torch.empty_like(x)
    bg.bg_packed_qk_norm_rope(x, x, None, torch.from_numpy(pos.astype(np.int32)).cuda(), q, k,
                              inv_freq=torch.from_numpy(freq).cuda(), interleaved=interleaved)
    assert torch.equal(q, k)
    got = q.double().cpu().numpy()[:, 0]
    got = got.reshape(len(pos), half, 2) if interleaved else np.stack((got[:, :half], got[:, half:]), -1)
    want = np.stack((np.cos(angle), np.sin(angle)), -1)
    e = off + 2.0 ** -21
    err = np.abs(got[rows, cols] - want) - (e + 2.0 ** -8 * (np.abs(want) + e))
    assert (err <= 0).all(), err.max()
