"""The few-row kernel of the window attention where test_gpu_window.py does not go: d = 64 with keys
that many CTAs share, tiles for several rounds of CTAs, windows as long as the table, and the weights'
sum.  Tolerances: test_gpu_window.py."""

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
@pytest.mark.parametrize("T,chunk", [(60, 0), (700, 0), (4000, 0), (4000, 512)])
def test_mean_of_equal_values(D, T, chunk):
    """Values that are the same for every key come out as they are.

    A key in sixteen (in every step of every warp) has weight 1, the others 2^-1 1.0037, which bf16
    rounds to 2^-1.  Divided by the sum of the weights as rounded, the mean of equal values is off by
    the rounding of sums of up to T fp32 terms, T 2^-23 < 2^-11 relative, and the rounding to bf16
    takes that back: the nearest numbers to a power of two are 2^-8 of it away.  Divided by the
    unrounded sum the mean is too small by 15 0.5 0.0037 / 8.53 = 0.0033, more than half of 2^-8, and
    comes out as the next number below."""
    H, Hk = 8, 2
    g = np.random.default_rng(T)
    value = torch.from_numpy(2.0 ** g.integers(-3, 4, (Hk, D)) * g.choice([-1, 1], (Hk, D))).to(torch.bfloat16).cuda()
    v = value.expand(1, T, Hk, D).contiguous()
    q = torch.zeros((1, 1, H, D), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, T, Hk, D), dtype=torch.bfloat16, device="cuda")
    # the others' logit, as a sum of bf16 numbers over the row's elements
    logit = float(np.log(0.5 * 1.0037))
    rest = logit
    for e in range(4):
        part = float(torch.tensor(rest).to(torch.bfloat16))
        q[..., e], k[..., e] = 1.0, part
        rest -= part
    k[0, ::16] = 0.0
    out, lse = run(q, k, v, T, 0, scale=1.0, opts=stl.options(key_chunk=chunk) if chunk else None)
    assert torch.equal(out.view(Hk, H // Hk, D), value[:, None].expand(Hk, H // Hk, D))
    # ex2 and log2 are off by 2^-22, the sum by T 2^-24
    ones = -(-T // 16)
    assert (lse.double() - np.log(ones + (T - ones) * np.exp(logit))).abs().max() < 2.0 ** -20 + T * 2.0 ** -24 + 2.0 ** -22 * 9


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
