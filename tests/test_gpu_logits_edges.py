"""GPU edges of bg_adjust_logits: penalties at and past the ends of their range, an index of no masks."""
import math

import numpy as np
import pytest

from tests import test_gpu_logits as tl

from attention_packed_varlen_causal_gb300 import binding as bg
from attention_packed_varlen_causal_gb300 import build
from oracle import logits as olg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    bg.load()


def lists(own_room, V, rows, groups):
    """Prompt tokens of each group and own tokens of each row, few (registers) or with room for many (counted)."""
    prompt = [[1, V - 1, 40 + g] for g in range(groups)]
    own = [[2, 2, (7 * i) % V] for i in range(rows)]
    table = np.zeros((rows, own_room), np.int64)
    table[:, :3] = own
    t = dict(own_tokens=tl.i32(table.tolist()).view(rows, own_room), own_lens=tl.i32([3] * rows))
    t["prompt_tokens"], t["cu_prompt"] = tl.packed(prompt)
    return dict(prompts=prompt, own=own), t


@pytest.mark.parametrize("own_room", [3, 60])
@pytest.mark.parametrize("V", [70, 4500])
def test_penalties_without_a_normal_reciprocal(V, own_room):
    """Their groups are left as they were and reported; the others are written."""
    import torch
    bad = [1e-39, 1e-45, 0.0, -0.0, -1.5, 3e38, math.inf, -math.inf, math.nan]
    fine = [1.5, 2.0 ** -126, 2.0 ** 126]
    rep = np.array(bad[:5] + fine + bad[5:], np.float32)
    G, per = len(rep), 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((G * per, V), generator=gen, device="cuda")
    h, t = lists(own_room, V, G * per, G)
    out, st = torch.full_like(x, tl.GUARD), tl.i32([0])
    kw = dict(t, rows_per_group=per)
    bg.bg_adjust_logits(x, out, repetition=torch.from_numpy(rep).cuda(), dev_status=st, **kw)
    assert int(st.item()) == bg.BG_DEVSTAT_PENALTY
    rows = [i for i in range(G * per) if 5 <= i // per < 8]
    rest = [i for i in range(G * per) if i not in rows]
    assert (out[rest] == tl.GUARD).all() and (out[rows] != tl.GUARD).all()
    want, st = torch.empty_like(x), tl.i32([0])
    rep[:5] = rep[8:] = 1.0
    bg.bg_adjust_logits(x, want, repetition=torch.from_numpy(rep).cuda(), dev_status=st, **kw)
    assert int(st.item()) == 0 and torch.equal(out[rows], want[rows])


@pytest.mark.parametrize("own_room", [3, 60])
@pytest.mark.parametrize("types", tl.TYPES, ids="-".join)
def test_penalties_at_the_ends_of_their_range(types, own_room):
    """Factors next to 2^-126 and 2^126, of logits whose products and quotients are normal numbers."""
    import torch
    V, per = 1100, 2
    rep = np.array([1.3 * 2.0 ** -126, 0.7 * 2.0 ** 126, 1.0, 1.0 + 2.0 ** -23, 3.0], np.float32)
    G = len(rep)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.rand((G * per, V), generator=gen, device="cuda") * 1.4 + 1.5
    x = torch.where(torch.rand(x.shape, generator=gen, device="cuda") < 0.5, x, -x).to(getattr(torch, types[0]))
    h, t = lists(own_room, V, G * per, G)
    out, st = torch.empty(x.shape, dtype=getattr(torch, types[1]), device="cuda"), tl.i32([0])
    bg.bg_adjust_logits(x, out, rows_per_group=per, repetition=torch.from_numpy(rep).cuda(), dev_status=st, **t)
    assert int(st.item()) == 0
    tl.assert_close(out, olg.adjust(x.double().cpu().numpy(), per, repetition=rep, **h), types[1] == "bfloat16")


@pytest.mark.parametrize("own_room", [3, 60])
@pytest.mark.parametrize("V", [70, 4500])
def test_no_masks_at_all(V, own_room):
    """A step none of whose rows has a grammar: an empty set of masks (or none) and an index of -1 change nothing; any other
    index is reported and its row left as it was."""
    import torch
    G, per = 3, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((G * per, V), generator=gen, device="cuda")
    h, t = lists(own_room, V, G * per, G)
    kw = dict(t, rows_per_group=per, repetition=torch.full((G,), 1.25, device="cuda"))
    want = torch.empty_like(x)
    bg.bg_adjust_logits(x, want, **kw)
    for mask in (torch.empty((0, (V + 31) // 32), dtype=torch.int32, device="cuda"), None):
        index = tl.i32([-1] * (G * per))
        out, st = torch.full_like(x, tl.GUARD), tl.i32([0])
        bg.bg_adjust_logits(x, out, mask=mask, mask_index=index, dev_status=st, **kw)
        assert int(st.item()) == 0 and torch.equal(out, want)
        for bad in (0, -2, 1 << 30):
            index[3] = bad
            out, st = torch.full_like(x, tl.GUARD), tl.i32([0])
            bg.bg_adjust_logits(x, out, mask=mask, mask_index=index, dev_status=st, **kw)
            rest = [0, 1, 2, 4, 5]
            assert int(st.item()) == bg.BG_DEVSTAT_MASK and (out[3] == tl.GUARD).all() and torch.equal(out[rest], want[rest])
