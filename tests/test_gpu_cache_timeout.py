"""The bounded waits of the 128-row attention kernels: a load that never comes makes a wait expire, the
call reports it, and the device goes on working."""

from __future__ import annotations

import pytest
import torch

import streaming_top_lightning_b200 as stl
from tests import test_gpu_cache4 as tc, test_gpu_window as tw

pytestmark = pytest.mark.gpu


def test_window_tiles_time_out():
    q, k, v = tw.inputs(2, 100, 300, 8, 2, 128, seed=1)
    want = stl.window_attention(q, k, v, 64, 4)
    assert stl.device_error() == 0
    stl.window_attention(q, k, v, 64, 4, opts=stl.options(timeout_ms=20, debug_flags=1))
    assert stl.device_error() == -7
    got = stl.window_attention(q, k, v, 64, 4)
    assert stl.device_error() == 0 and torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("B", [1, 200])  # clusters that join a tile's chunks; a CTA a tile, several each
def test_cache4_tiles_time_out(B):
    c = tc.Filled(1, 600, 1, 128, 16, seed=2)
    pages, table = c.on_gpu()
    table = table.expand(B, -1).contiguous()
    q = tc.queries(B, 1, 64, 128, seed=3)
    lens = tc.dev([600] * B)
    want = stl.cache4_attention(q, pages, table, lens, 1, 16)
    assert stl.device_error() == 0
    stl.cache4_attention(q, pages, table, lens, 1, 16, opts=stl.options(timeout_ms=20, debug_flags=1))
    assert stl.device_error() == -7
    got = stl.cache4_attention(q, pages, table, lens, 1, 16)
    assert stl.device_error() == 0 and torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
