"""The pages' life on the GPU against a Python model, call by call: every table, count, length and
byte has to be equal."""

from __future__ import annotations

import random

import numpy as np
import pytest
import torch

import streaming_top_lightning_b200 as stl
from tests import _cache

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """The same pool on the GPU and in the model."""

    def __init__(self, B, width, n, page, size, seed=0):
        g = np.random.default_rng(seed)
        content = g.integers(0, 256, (n, size), dtype=np.uint8)
        self.m = _cache.Pool([0] * n, [[-1] * width for _ in range(B)], [0] * B, page, content.copy())
        self.page = page
        self.pages = torch.from_numpy(content).cuda()
        self.refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def same(self):
        assert self.refs.tolist() == self.m.refs
        assert self.table.tolist() == self.m.table
        assert self.lens.tolist() == self.m.lens
        assert np.array_equal(self.pages.cpu().numpy(), self.m.content)

    def grow(self, lens):
        got = stl.cache_extend(self.refs, self.table, dev(lens), self.page)
        assert got.tolist() == [self.m.extend(lens)]
        self.lens.copy_(dev(lens))
        self.m.lens = list(lens)
        self.same()

    def free(self, rows):
        stl.cache_free(self.refs, self.table, self.lens, dev(rows))
        self.m.free(rows)
        self.same()

    def fork(self, src, dst):
        got = stl.cache_fork(self.pages, self.refs, self.table, self.lens, dev(src), dev(dst), self.page)
        assert got.tolist() == [self.m.fork(src, dst)]
        self.same()

    def compact(self, in_place):
        out = (self.table, self.refs) if in_place else None
        table, refs, live = stl.cache_compact(self.pages, self.refs, self.table, out=out)
        assert live.tolist() == [self.m.compact()]
        self.table, self.refs = table, refs
        self.same()


@pytest.mark.parametrize("B,width,n,page,size", [(1, 1, 1, 1, 16), (5, 7, 40, 16, 48), (40, 33, 500, 4, 16400), (70, 9, 5000, 64, 160)])
def test_a_life(B, width, n, page, size):
    """Random growth, forks, ends and compactions; pools that run out on the way."""
    r = random.Random(n)
    p = Both(B, width, n, page, size, seed=n)
    for step in range(12):
        p.grow([min(width * page, x + r.choice([0, 1, page, 3 * page + 1])) for x in p.m.lens])
        if step % 3 == 1:
            p.m.lens = [min(x, page * sum(e >= 0 for e in row)) for x, row in zip(p.m.lens, p.m.table)]
            p.lens.copy_(dev(p.m.lens))
        p.free([r.randrange(B) for _ in range(B // 2)])
        empty = [b for b in range(B) if p.m.lens[b] == 0]
        r.shuffle(empty)
        p.fork([r.randrange(B) for _ in empty], empty)
        if step % 4 == 3:
            p.compact(step % 8 == 3)


def test_refused_children():
    p = Both(8, 4, 30, 16, 32)
    p.grow([40, 0, 16, 0, 0, 0, 64, 5])
    # out of range, onto itself, an occupied row, one row twice, a parent that is empty, a chain
    p.fork([0, -1, 0, 8, 0, 0, 2, 1, 0, 6, 3], [1, 3, 8, 3, 0, 2, 3, 4, 3, 5, 1])
    # a length beyond the row, and a last page that is not there
    p.free([1, 3, 4, 5])
    p.lens[0], p.m.lens[0] = 65, 65
    p.table[7, 0], p.m.table[7][0] = -1, -1
    p.fork([0, 7, 2], [1, 3, 4])


def test_free_skips_and_repeats():
    p = Both(4, 3, 10, 8, 16)
    p.grow([24, 8, 1, 0])
    p.fork([0], [3])
    p.free([0, 0, -1, 4, 2, 2, 0, 3])
    p.free([])


def test_pool_runs_out_in_order():
    p = Both(3, 4, 5, 2, 16)
    p.grow([3, 8, 4])     # 2 + 3 pages: the last row gets none
    p.free([0])
    p.m.lens[2] = 0
    p.lens[2] = 0
    p.grow([0, 8, 4])


def test_large_pool():
    """More pages than a cluster's threads take at once, ranks far apart."""
    p = Both(300, 200, 70000, 16, 16, seed=3)
    r = random.Random(3)
    p.grow([r.randrange(0, 3200) for _ in range(300)])
    p.free([r.randrange(300) for _ in range(150)])
    p.compact(False)
    p.grow([max(x, r.randrange(0, 3200)) for x in p.m.lens])


def test_compact_keeps_odd_entries():
    """Entries that name a free page become -1, those outside the pool stay."""
    p = Both(2, 4, 12, 4, 16)
    p.grow([16, 16])
    p.free([0])
    p.table[0, 0], p.m.table[0][0] = 2, 2
    p.table[0, 1], p.m.table[0][1] = 99, 99
    p.compact(True)


def test_graph():
    """A captured step: end, fork, grow; replayed against the model."""
    B, width, page = 8, 6, 4
    p = Both(B, width, 60, page, 64)
    p.grow([5, 7, 12, 1, 0, 0, 0, 0])
    src, dst = dev([0, 1, 2, 3]), dev([4, 5, 6, 7])
    lens = p.lens.clone()
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")

    def step():
        stl.cache_free(p.refs, p.table, p.lens, dst)
        stl.cache_fork(p.pages, p.refs, p.table, p.lens, src, dst, page, workspace=ws)
        torch.add(p.lens, 1, out=lens)
        stl.cache_extend(p.refs, p.table, lens, page, workspace=ws)

    def model():
        p.m.free([4, 5, 6, 7])
        p.m.fork([0, 1, 2, 3], [4, 5, 6, 7])
        p.m.extend([x + 1 for x in p.m.lens])

    step()
    model()
    p.same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    p.same()
    for _ in range(3):
        graph.replay()
        model()
        p.same()
