"""The plain implementations that the cache tests compare with, checked themselves on the CPU."""

from __future__ import annotations

import random
from fractions import Fraction

import numpy as np
import torch

from tests import _cache


def test_number_tables():
    assert _cache.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, _cache.E4M3)


def test_rounding_against_torch():
    g = np.random.default_rng(0)
    x = np.abs(g.standard_normal(50000)).astype(np.float32) * 60
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(_cache.E4M3[_cache.nearest(x, _cache.E4M3)], want)
    y = (g.standard_normal(50000) * 10.0 ** g.integers(-30, 30, 50000)).astype(np.float32)
    assert np.array_equal(_cache.bf16(y), torch.from_numpy(y).to(torch.bfloat16).double().numpy())


def test_ties_go_to_even():
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert _cache.E2M1[_cache.nearest(mids, _cache.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4]


def test_quantise_by_fractions():
    """Blocks by exact fractions: the nearest scale, then the nearest codes, where fp32 is exact."""
    g = np.random.default_rng(1)
    x = _cache.bf16(g.standard_normal((20, 32)) * 3)
    code, sc = _cache.quantise(x, 1.0)
    for row in range(20):
        for b in range(2):
            blk = [Fraction(float(v)) for v in x[row, 16 * b:16 * b + 16]]
            top = max(abs(v) for v in blk) / 6
            dist = [abs(Fraction(float(n)) - top) for n in _cache.E4M3]
            assert dist[sc[row, b]] <= min(dist) + Fraction(1, 10 ** 7)
            s = Fraction(float(_cache.E4M3[sc[row, b]]))
            for v, c in zip(blk, code[row, 16 * b:16 * b + 16]):
                d = [abs(Fraction(float(n)) * s - min(abs(v), 6 * s)) for n in _cache.E2M1]
                assert d[c & 7] == min(d) and (v >= 0 or c & 8)


def test_attend_is_softmax():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal(8), g.standard_normal((5, 8)), g.standard_normal((5, 8))
    o, a, lse, _ = _cache.attend(q, k, v, 0.5)
    w = np.exp(k @ q * 0.5)
    assert np.allclose(o, w @ v / w.sum()) and np.allclose(lse, np.log(w.sum())) and np.all(a >= np.abs(o) - 1e-12)
    assert _cache.attend(q, k[:0], v[:0], 0.5)[2] == -np.inf


def test_pool_invariants():
    """Every page's count is the number of rows that hold it, whatever the calls."""
    r = random.Random(3)
    n, B, width, page = 40, 9, 6, 4
    p = _cache.Pool([0] * n, [[-1] * width for _ in range(B)], [0] * B, page, np.arange(n * 16).reshape(n, 16))
    for _ in range(300):
        what = r.choice(["grow", "free", "fork", "compact"])
        if what == "grow":
            p.extend(lens := [min(width * page, x + r.randrange(4)) for x in p.lens])
            p.lens = [min(x, page * sum(e >= 0 for e in row)) for x, row in zip(lens, p.table)]
        elif what == "free":
            p.free([r.randrange(-1, B + 1) for _ in range(3)])
        elif what == "fork":
            before = {b: [p.content[e].copy() for e in p.table[b] if e >= 0] for b in range(B)}
            src, dst = [r.randrange(B) for _ in range(3)], [r.randrange(B) for _ in range(3)]
            was = list(p.lens)
            p.fork(src, dst)
            for s, d in zip(src, dst):
                if s != d and was[d] == 0 and p.lens[d] and was[s] == p.lens[d]:
                    held = -(-p.lens[d] // page)
                    assert any(all(np.array_equal(p.content[e], c) for e, c in zip(p.table[d], before[x])) for x in src
                               if len(before[x]) >= held)
        else:
            was = [[p.content[e].copy() for e in row if e >= 0] for row in p.table]
            live = p.compact()
            assert all(x > 0 for x in p.refs[:live]) and not any(p.refs[live:])
            for row, c in zip(p.table, was):
                assert all(np.array_equal(p.content[e], x) for e, x in zip([e for e in row if e >= 0], c))
        held = [e for row in p.table for e in row if e >= 0]
        assert [held.count(i) for i in range(n)] == p.refs
