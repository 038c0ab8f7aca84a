"""The few-row kernel of the window attention where test_gpu_window.py does not go: d = 64 with keys
that many CTAs share, tiles for several rounds of CTAs.  Tolerances: test_gpu_window.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import streaming_top_lightning_b200 as stl
from tests.test_gpu_window import check, inputs, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hk", [(8, 2), (12, 1), (24, 8)])
@pytest.mark.parametrize("chunk", [0, 128, 640])
def test_d64_shares(H, Hk, chunk):
    """Ragged sequences whose keys the CTAs of one wave share, d = 64."""
    B, T = 9, 3100
    q, k, v = inputs(B, 1, T, H, Hk, 64, seed=H + chunk)
    lens = [T, 0, 1, 33, 64, 700, 1999, T - 1, 2500]
    out, lse = run(q, k, v, T, 4, lens, [1, 1, 1, 0, 1, 1, 1, 1, 1], opts=stl.options(key_chunk=chunk) if chunk else None)
    check(q, k, v, T, 4, lens, [1, 1, 1, 0, 1, 1, 1, 1, 1], out, lse, fill=7.0)


@pytest.mark.parametrize("D", [64, 128])
def test_several_rounds_of_ctas(D):
    """Tiles for one and a half times the places, each a CTA of its own."""
    B, T, H, Hk = 56, 900, 8, 8
    q, k, v = inputs(B, 1, T, H, Hk, D, seed=D + 1)
    g = np.random.default_rng(D)
    lens = [int(x) for x in g.integers(0, T + 1, B)]
    out, lse = run(q, k, v, 200, 4, lens, [1] * B)
    check(q, k, v, 200, 4, lens, [1] * B, out, lse, rows={(b, 0) for b in range(0, B, 5)})
