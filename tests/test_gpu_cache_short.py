"""Sequences of a few tokens in the attention kernels' 128-row tiles: fewer keys than a TMA box, a
block or a page, more query rows than tokens.  Tolerances: test_gpu_window.py and test_gpu_cache4.py;
the window's weights are divided by the sum of the weights as rounded, which makes 2^-8 (a + |o|) of
their 2^-8 a."""

from __future__ import annotations

import pytest
import torch

from tests import test_gpu_cache4 as tc
from tests import test_gpu_window as tw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 31, 33])
@pytest.mark.parametrize("S,H,Hk", [(1, 32, 1), (3, 128, 2), (40, 3, 3), (17, 1, 1)])
def test_window(S, H, Hk, T, D):
    B = 3
    q, k, v = tw.inputs(B, S, T, H, Hk, D, seed=S + T)
    for window, sinks, lens, q_lens in ((T, 0, [T] * B, [min(S, T)] * B), (1, 1, [T, 1, 0], [S, S, min(S, 2)])):
        out, lse = tw.run(q, k, v, window, sinks, lens, q_lens)
        tw.check(q, k, v, window, sinks, lens, q_lens, out, lse, u=2 * tw.U_BF16, fill=7.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 17, 33])
@pytest.mark.parametrize("S,H,Hk", [(1, 17, 1), (1, 32, 1), (2, 64, 4), (40, 3, 3)])
def test_cache4(S, H, Hk, T, D):
    B = 3
    c = tc.Filled(B, T, Hk, D, 16, seed=T)
    q = tc.queries(B, S, H, D, seed=S + T)
    for window, sinks, lens, q_lens in ((0, 0, [T] * B, [min(S, T)] * B), (1, 1, [T, 1, 0], [S, S, min(S, 2)])):
        out, lse = tc.attend(c, q, lens, q_lens, window, sinks)
        tc.check(c, q, window, sinks, lens, q_lens, out, lse)


@pytest.mark.parametrize("H,topk", [(17, 1), (32, 5), (24, 100), (100, 33)])
def test_listed(H, topk):
    """Few entries, repeated ones among them, and rows that list nothing."""
    B, S, T = 2, 3, 50
    c = tc.Filled(B, T, 1, 128, 16, seed=H)
    q = tc.queries(B, S, H, 128, seed=topk)
    idx = torch.randint(0, T, (B, S, topk), generator=torch.Generator().manual_seed(topk), dtype=torch.int32).numpy()
    idx[0, 1] = -1
    idx[1, 0, :topk // 2] = T + 3  # past the sequence's end
    out, lse = tc.attend(c, q, [T, T], [S, S], idx=idx)
    tc.check(c, q, 0, 0, [T, T], [S, S], out, lse, see=lambda b, i: idx[b, i][(idx[b, i] >= 0) & (idx[b, i] < T)])
