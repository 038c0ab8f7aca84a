"""The few-row kernel of the window attention where test_gpu_window.py does not go: d = 64 with keys
that many CTAs share, tiles for several rounds of CTAs, windows as long as the table.  Tolerances: test_gpu_window.py."""

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


@pytest.mark.parametrize("D,T", [(64, 20000), (128, 9000)])
def test_ragged_under_a_long_window(D, T):
    """A tile for each of the places, a window as long as the table: ragged sequences share the CTAs,
    and without lengths each tile has one and needs no workspace."""
    B, H, Hk = 37, 16, 8
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((B, 1, H, D), (B, T, Hk, D), (B, T, Hk, D)))
    lens = [T, 0, 1] + [int(x) for x in np.random.default_rng(D).integers(0, T, B - 3)]
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    with pytest.raises(stl.StreamIndexError):
        run(q, k, v, T, 0, lens, workspace=none)
    for n, (out, lse) in ((lens, run(q, k, v, T, 0, lens)), ([T] * B, run(q, k, v, T, 0, workspace=none))):
        for b in (0, 1, 2, 7, B - 1):
            one = slice(b, b + 1)
            check(q[one], k[one], v[one], T, 0, n[one], [1], out[one], lse[one])


@pytest.mark.parametrize("D", [64, 128])
def test_several_rounds_of_ctas(D):
    """Tiles for one and a half times the places, each a CTA of its own."""
    B, T, H, Hk = 56, 900, 8, 8
    q, k, v = inputs(B, 1, T, H, Hk, D, seed=D + 1)
    g = np.random.default_rng(D)
    lens = [int(x) for x in g.integers(0, T + 1, B)]
    out, lse = run(q, k, v, 200, 4, lens, [1] * B)
    check(q, k, v, 200, 4, lens, [1] * B, out, lse, rows={(b, 0) for b in range(0, B, 5)})
