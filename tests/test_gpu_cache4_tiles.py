"""The 4-bit cache's attention in 128-row tiles (17 rows of a kv head and more) where the few-row tests of
test_gpu_cache4.py do not reach: tables that name no page, and queries outside fp16's range.  Tolerances:
test_gpu_cache4.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import _cache, test_gpu_cache4 as tc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,H,Hk,D", [(2, 4, 1, 64), (2, 32, 1, 64), (1, 128, 1, 128), (3, 64, 2, 128), (30, 8, 2, 64)])
@pytest.mark.parametrize("kind", ["whole", "window", "listed"])
def test_missing_pages_are_not_attended(S, H, Hk, D, kind):
    """Entries that are free, past the pool's end or negative, among the first, the last and between."""
    T, n, page = 256, 250, 16
    c = tc.Filled(1, T, Hk, D, page, seed=4)
    q = tc.queries(1, S, H, D, seed=4)
    gone = {0: -1, 3: -1, 7: 10 ** 6, 8: c.pages.shape[0], 12: -5, 13: 2 ** 31 - 1, 15: -2 ** 31}
    for e, pg in gone.items():
        c.table[0, e] = pg
    away = [j for e in gone for j in range(page * e, page * e + page)]
    window, sinks, idx = (60, 20, None) if kind == "window" else (0, 0, None)
    if kind == "listed":
        idx = np.random.default_rng(S).integers(-1, T, (1, S, 100)).astype(np.int32)
        idx[0, S // 2, 50:] = away[3]
    out, lse = tc.attend(c, q, [n], [S], window, sinks, idx=idx)

    def see(b, i):
        if idx is not None:
            return np.array([j for j in idx[b, i] if 0 <= j < n and j not in away], int)
        return np.setdiff1d(np.flatnonzero(_cache.visible(n - S + i, n, window, sinks)), away)

    tc.check(c, q, window, sinks, [n], [S], out, lse, see=see)
    c.table[:] = -1
    out, lse = tc.attend(c, q, [n], [S], window, sinks, idx=idx)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("H,D", [(4, 64), (32, 128), (128, 64), (200, 128)])
def test_query_range(H, D):
    """Queries far outside fp16's range, both ways, and rows of zeros."""
    c = tc.Filled(1, 200, 1, D, 16, seed=8)
    q = tc.queries(1, 4, H, D, seed=8)
    q[0, 0] *= 2.0 ** 60
    q[0, 1] *= 2.0 ** -60
    q[0, 2] = 0
    q[0, 3, 0, 5] = 2.0 ** 40
    for i, scale in ((0, 2.0 ** -63), (1, 2.0 ** 56), (2, 0.1), (3, 2.0 ** -43)):
        out, lse = tc.attend(c, q, [200], [4], scale=scale)
        assert torch.isfinite(out[0, i]).all()
        tc.check(c, q, 0, 0, [200], [4], out, lse, scale=scale, rows={(0, i)})
