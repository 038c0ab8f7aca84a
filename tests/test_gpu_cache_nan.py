"""NaN scales in a 4-bit cache that some rows see and others do not.  Tolerances:
test_gpu_window.py and test_gpu_cache4.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import streaming_top_lightning_b200 as stl
from tests import _cache, test_gpu_cache4 as tc

pytestmark = pytest.mark.gpu


def scale_bytes(c, j, h, is_v):
    """The scale bytes of sequence 0's token j, a view."""
    return c.cache._at(c.table[0, j // c.page], h, j % c.page, is_v)[1]


@pytest.mark.parametrize("S,H,Hk,D", [(3, 4, 2, 64), (3, 4, 2, 128), (4, 12, 3, 128), (9, 24, 3, 128), (9, 24, 3, 64), (50, 4, 2, 128),
                                      (130, 2, 2, 64)])
@pytest.mark.parametrize("window,chunk", [(0, 0), (60, 0), (0, 128)])
@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_nan_scales(S, H, Hk, D, window, chunk, code):
    """A NaN scale reaches the rows that see its key, there its 16 elements alone, and no other row."""
    T, page = 300, 16
    c = tc.Filled(1, T, Hk, D, page, seed=S + D)
    t0 = T - S
    late, mid = T - 2, t0 + S // 2           # seen by the queries from their own on
    early = t0 - window + 1 if window else 2  # seen by the first query alone, or by all
    blocks = {late: [0], mid: [D // 16 - 1, 1], early: [2]}
    for j, bad in blocks.items():
        for h in range(Hk):
            scale_bytes(c, j, h, True)[bad] = code
    q = tc.queries(1, S, H, D, seed=S)
    out, lse = tc.attend(c, q, [T], [S], window, 4 if window else 0, opts=stl.options(key_chunk=chunk) if chunk else None)
    want = torch.zeros((S, D // 16), dtype=torch.bool)
    for i in range(S):
        for j, bad in blocks.items():
            if _cache.visible(t0 + i, T, window, 4)[j]:
                want[i, bad] = True
    nan = torch.isnan(out[0].cpu()).view(S, H, D // 16, 16)
    assert torch.equal(nan, want[:, None, :, None].expand(S, H, D // 16, 16))
    assert torch.isfinite(lse).all()
    # everything else by the formula over the numbers that the codes stand for (the scales before)
    ref = out.clone()
    some = {(0, i) for i in {0, 1, S // 2 - 1, S // 2, S - 2, S - 1}}
    for _, i in some:
        for h in range(H):
            sel = np.flatnonzero(_cache.visible(t0 + i, T, window, 4))
            o = _cache.attend(q[0, i, h].double().cpu().numpy(), c.kv[0][0, sel, h * Hk // H].numpy(), c.kv[1][0, sel, h * Hk // H].numpy(),
                              D ** -0.5)[0]
            ref[0, i, h] = torch.where(torch.isnan(out[0, i, h].cpu()), torch.from_numpy(o).to(torch.bfloat16), out[0, i, h].cpu()).cuda()
    tc.check(c, q, window, 4 if window else 0, [T], [S], ref, lse, rows=some)


@pytest.mark.parametrize("S,H,Hk", [(3, 4, 2), (9, 24, 3)])
def test_nan_key_scales(S, H, Hk):
    """A NaN key scale: NaN rows where the key is seen, nothing elsewhere."""
    T = 200
    c = tc.Filled(1, T, Hk, 128, 16, seed=S)
    for h in range(Hk):
        scale_bytes(c, T - 2, h, False)[3] = 0x7F
    q = tc.queries(1, S, H, 128, seed=S)
    out, lse = tc.attend(c, q, [T], [S])
    assert torch.isnan(out[0, S - 2:]).all() and torch.isnan(lse[0, S - 2:]).all()
    tc.check(c, q, 0, 0, [T], [S], out, lse, rows={(0, i) for i in range(S - 2)})
