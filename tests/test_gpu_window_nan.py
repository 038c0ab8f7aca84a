"""Window attention over infinities and NaN in values that some rows see and others do not.  Tolerances:
test_gpu_window.py and, for rows whose keys several chunks hold, test_gpu_window_chunks.py."""

from __future__ import annotations

import pytest
import torch

import streaming_top_lightning_b200 as stl
from tests import test_gpu_window as tw

pytestmark = pytest.mark.gpu


def test_recomputed_rows_and_the_waits_clock():
    """One CTA goes through a prompt whose values hold a NaN in the middle of a tile: the rows before
    it are computed again, which takes longer than a wait may, and the items after it still come out."""
    S, H, Hk, D = 3000, 8, 1, 64
    q, k, v = tw.inputs(1, S, S, H, Hk, D, seed=1)
    bad = 1999
    v[0, bad, 0, 7] = float("nan")
    out, lse = tw.run(q, k, v, S, 0, opts=stl.options(grid_ctas=1, timeout_ms=3))
    nan = torch.isnan(out[0])
    assert not nan[:bad].any() and nan[bad:, :, 7].all()
    nan[bad:, :, 7] = False
    assert not nan.any() and torch.isfinite(lse).all()
    rows = {(0, i) for i in (bad - 14, bad - 1)}
    tw.check(q, k, torch.nan_to_num(v), S, 0, [S], [S], out, lse, rows=rows)


@pytest.mark.parametrize("D,H,Hk", [(64, 8, 2), (128, 8, 1), (128, 2, 2)])
@pytest.mark.parametrize("S,T,window", [(400, 400, 100), (40, 4000, 3000)])
def test_values_around_the_sinks(D, H, Hk, S, T, window):
    """Values just behind the sinks, which share their block, and values of the sinks themselves."""
    sinks, t0 = 5, T - S
    q, k, v = tw.inputs(1, S, T, H, Hk, D, seed=S)
    behind = v.clone()
    behind[0, sinks:31] = float("nan")
    out, lse = tw.run(q, k, behind, window, sinks)
    # rows from here on see none of them
    free = max(0, 31 + window - t0 - 1)
    assert torch.isfinite(out[0, free:]).all() and torch.isfinite(lse).all()
    tw.check(q, k, v, window, sinks, [T], [S], out, lse, u=2 * tw.U_BF16, rows={(0, i) for i in (free, (free + S) // 2, S - 1)})
    v[0, 2, :, 9] = float("nan")
    v[0, 3, :, 11] = float("inf")
    out, lse = tw.run(q, k, v, window, sinks)
    seen = torch.arange(S) + t0
    assert torch.equal(torch.isnan(out[0, :, :, 9]).all(1).cpu(), seen >= 2) and torch.equal(torch.isposinf(out[0, :, :, 11]).all(1).cpu(), seen >= 3)
    out[0, :, :, 9], out[0, :, :, 11] = 0, 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("S", [6, 100])
def test_infinite_values_beside_unseen_nan(S):
    """Rows that see an infinity keep it where a key that they do not see holds a NaN."""
    T, window = 300, 50
    q, k, v = tw.inputs(1, S, T, 4, 2, 128, seed=S)
    v[0, T - S - 10, :, 3] = float("inf")
    v[0, T - S - 20, :, 4] = float("nan")
    v[0, T - 1] = float("nan")
    out, lse = tw.run(q, k, v, window, 0)
    for i in range(S - 1):
        t = T - S + i
        assert torch.isposinf(out[0, i, :, 3]).all() == (T - S - 10 > t - window), i
        assert torch.isnan(out[0, i, :, 4]).all() == (T - S - 20 > t - window), i
    out[..., 3], out[..., 4] = 0, 0
    assert torch.isfinite(out[0, :-1]).all() and torch.isnan(out[0, -1, :, 5]).all()


@pytest.mark.parametrize("S", [4, 200])
def test_values_that_are_all_nan(S):
    q, k, v = tw.inputs(1, S, 500, 8, 2, 64, seed=S)
    v[:] = float("nan")
    out, lse = tw.run(q, k, v, 100, 4)
    assert torch.isnan(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("H", [2, 40])
@pytest.mark.parametrize("S,T,window,sinks", [(65, 65, 20, 60), (9, 65, 59, 68), (40, 3000, 2500, 700)])
def test_infinite_values_in_both_blocks(H, S, T, window, sinks):
    """A key behind the first sinks in their block and again in the window's: an infinity that a row
    sees there is its result, whatever the masked columns make of it."""
    q, k, v = tw.inputs(1, S, T, H, 1, 64, seed=S)
    bad = [min(10, sinks - 1), min(30, sinks - 1), T - S // 2]
    for e, j in enumerate(bad):
        v[0, j, 0, e] = float("inf") if e % 2 else float("-inf")
    out, lse = tw.run(q, k, v, window, sinks)
    assert torch.isfinite(lse).all()
    t = torch.arange(T - S, T)
    for e, j in enumerate(bad):
        sees = (t >= j) & ((t - j < window) | (j < sinks))
        assert torch.equal(torch.isinf(out[0, :, :, e]).cpu(), sees[:, None].expand(S, H)), (e, j)
        assert not torch.isnan(out[0, :, :, e]).any()
    out[..., :3] = 0
    assert torch.isfinite(out).all()
