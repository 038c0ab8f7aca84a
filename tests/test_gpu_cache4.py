"""The 4-bit paged cache on the GPU: rows in and out bit by bit, and its attention against 64-bit
rows over the numbers that the codes stand for.

Tolerance of the attention: as the window attention's, with 2^-11 for the rounding of a probability
to fp16 in place of bf16's 2^-8 (tests/test_gpu_window.py).  fp16 numbers below 2^-14 are multiples
of 2^-24: a probability, rounded after a scale of 2^10 (the row's largest so far being 2^10), is off
by at most 2^-25 2^-10 = 2^-35 of the largest besides, which is at most one, so an output by
2^-35 sum_j |v_j| besides.  Codes times block scales are exact in
fp16, and a query row is exact after its power of two but for elements below 2^-24 of its largest:
those add D 2^-25 of the largest |q| times |k| to a dot product, which the term for the sum's
rounding, doubled, covers."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import synth
import streaming_top_lightning_b200 as stl
from tests import _cache, _gpu, test_gpu_window as tw

pytestmark = pytest.mark.gpu

U_FP16 = torch.finfo(torch.float16).eps / 2


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


class Filled:
    """A cache with every page of every sequence written by the test's own quantiser."""

    def __init__(self, B, T, heads, dim, page, seed, k_scale=1.0, v_scale=1.0, spare=3):
        g = np.random.default_rng(seed)
        self.B, self.T, self.heads, self.dim, self.page = B, T, heads, dim, page
        self.g = (k_scale, v_scale)
        self.width = -(-T // page)
        n = B * self.width + spare
        self.table = g.permutation(n)[:B * self.width].reshape(B, self.width).astype(np.int32)
        # pages and slots that no token has hold NaN scales and any codes
        self.pages = g.integers(0, 256, (n, stl.cache4_page_bytes(heads, dim, page)), dtype=np.uint8)
        cache = _cache.Cache4(self.pages, heads, dim, page)
        for pg in range(n):
            for h in range(heads):
                base = h * cache.block + page * dim
                self.pages[pg, base:base + 2 * page * dim // 16] = 0x7F
        self.kv = []
        for is_v in (False, True):
            x = g.standard_normal((B, T, heads, dim)) * np.exp(g.standard_normal((B, T, heads, 1)))
            code, sc = _cache.quantise(_cache.bf16(x), self.g[is_v])
            for b in range(B):
                for j in range(T):
                    for h in range(heads):
                        cache.put(self.table[b, j // page], h, j % page, is_v, code[b, j, h], sc[b, j, h])
            self.kv.append(torch.from_numpy(_cache.values(code, sc, self.g[is_v])))
        self.cache = cache

    def on_gpu(self):
        return torch.from_numpy(self.pages).cuda(), dev(self.table)


def attend(c, q, lens, q_lens, window=0, sinks=0, idx=None, **kw):
    B, S, H, D = q.shape
    out = torch.full((B, S, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, S, H), 7.0, device="cuda")
    pages, table = c.on_gpu()
    stl.cache4_attention(q, pages, table, dev(lens), c.heads, c.page, window, sinks, q_lens=dev(q_lens),
                         idx=None if idx is None else dev(idx), k_scale=c.g[0], v_scale=c.g[1], out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert stl.device_error() == 0
    return out, lse


def queries(B, S, H, D, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, S, H, D), generator=g) * spread).to(torch.bfloat16).cuda()


def check(c, q, window, sinks, lens, q_lens, out, lse, **kw):
    return tw.check(q, c.kv[0], c.kv[1], window, sinks, lens, q_lens, out, lse, u=U_FP16, tiny=2.0 ** -35, fill=7.0,
                    **kw)


CASES = [
    # B, S, T, H, Hk, D, page, window, sinks
    (1, 1, 1, 1, 1, 64, 16, 0, 0),
    (2, 1, 100, 8, 2, 128, 16, 0, 0),
    (1, 1, 777, 4, 1, 64, 32, 0, 0),
    (1, 3, 300, 24, 8, 64, 64, 0, 0),
    (2, 1, 333, 128, 1, 128, 64, 0, 0),
    (1, 9, 150, 6, 2, 128, 128, 0, 0),
    (2, 1, 500, 8, 2, 128, 16, 100, 4),
    (1, 5, 400, 12, 12, 64, 256, 33, 61),
    (1, 40, 90, 4, 2, 128, 16, 0, 0),
]


@pytest.mark.parametrize("B,S,T,H,Hk,D,page,window,sinks", CASES)
def test_attention_against_formula(B, S, T, H, Hk, D, page, window, sinks):
    c = Filled(B, T, Hk, D, page, seed=T, k_scale=0.5, v_scale=2.0)
    q = queries(B, S, H, D, seed=T)
    out, lse = attend(c, q, [T] * B, [S] * B, window, sinks)
    check(c, q, window, sinks, [T] * B, [S] * B, out, lse)


def test_attention_ragged():
    B, S, T = 6, 4, 208
    c = Filled(B, T, 2, 64, 16, seed=1)
    q = queries(B, S, 6, 64, seed=2)
    lens, q_lens = [T, 0, 1, 17, 160, T + 99], [S, S, 2, 0, 3, S + 1]
    out, lse = attend(c, q, lens, q_lens)
    check(c, q, 0, 0, [min(n, T) for n in lens], [min(n, S) for n in q_lens], out, lse)


@pytest.mark.parametrize("H,Hk,D,page,topk", [(128, 1, 128, 64, 100), (8, 2, 64, 16, 37), (20, 4, 128, 32, 1), (16, 1, 64, 16, 300)])
def test_listed_entries(H, Hk, D, page, topk):
    """The indexer's rows: padding, entries past the end, rows that list nothing, entries listed twice."""
    B, S, T = 2, 3, 260
    c = Filled(B, T, Hk, D, page, seed=topk, v_scale=0.25)
    q = queries(B, S, H, D, seed=topk)
    g = np.random.default_rng(topk)
    idx = g.integers(-1, T, (B, S, topk)).astype(np.int32)
    idx[0, 1] = -1
    idx[1, 0, topk // 2:] = T + 7
    idx[1, 2, :] = idx[1, 2, 0]
    lens = [T, 200]
    out, lse = attend(c, q, lens, [S, 2], idx=idx)
    see = lambda b, i: np.array([j for j in idx[b, i] if 0 <= j < lens[b]], int)  # noqa: E731
    check(c, q, 0, 0, lens, [S, 2], out, lse, see=see)


def test_missing_pages_are_not_attended():
    """A table entry that names no page (evicted, or out of the pool) holds no keys."""
    c = Filled(1, 256, 1, 64, 16, seed=4)
    q = queries(1, 2, 4, 64, seed=4)
    c.table[0, 3], c.table[0, 7], c.table[0, 12] = -1, 10 ** 6, -5
    out, lse = attend(c, q, [250], [2])
    gone = [j for e in (3, 7, 12) for j in range(16 * e, 16 * e + 16)]
    see = lambda b, i: np.setdiff1d(np.arange(248 + i + 1), gone)  # noqa: E731
    check(c, q, 0, 0, [250], [2], out, lse, see=see)
    c.table[:] = -1
    out, lse = attend(c, q, [250], [2])
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("chunk", [128, 512])
def test_key_chunks(chunk):
    c = Filled(2, 1100, 1, 128, 64, seed=chunk)
    q = queries(2, 1, 5, 128, seed=chunk)
    out, lse = attend(c, q, [1100, 300], [1, 1], opts=stl.options(key_chunk=chunk))
    check(c, q, 0, 0, [1100, 300], [1, 1], out, lse)


def test_query_range():
    """Queries far outside fp16's range, both ways, and rows of zeros."""
    c = Filled(1, 64, 1, 128, 16, seed=8)
    q = queries(1, 4, 4, 128, seed=8)
    q[0, 0] *= 2.0 ** 60
    q[0, 1] *= 2.0 ** -60
    q[0, 2] = 0
    q[0, 3, 0, 5] = 2.0 ** 40
    for i, scale in ((0, 2.0 ** -63), (1, 2.0 ** 56), (2, 0.1), (3, 2.0 ** -43)):
        out, lse = attend(c, q, [64], [4], scale=scale)
        assert torch.isfinite(out[0, i]).all()
        check(c, q, 0, 0, [64], [4], out, lse, scale=scale, rows={(0, i)})


def test_append_bits():
    """Codes and scales of every kind of block, written where the table says and nowhere else."""
    B, S, heads, page, T = 3, 50, 2, 16, 96
    for dim in (64, 128):
        g = np.random.default_rng(dim)
        x = [g.standard_normal((B, S, heads, dim)) * 2.0 ** g.integers(-14, 10, (B, S, heads, 1)) for _ in range(2)]
        x[0][0, 0] = 0.0
        x[0][0, 1, 0, :16] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -6, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25]
        x[0][0, 1, 1, :16] = [12, 10, 7, 5, 3.5, 2.5, 1.5, 0.5, 0, -0.0, 1e-3, -1e-3, 11, 9, 8, 6.5]
        x[1][0, 2, 0, :16] = 2.0 ** -12
        x[1][0, 3] = 3e38
        x[1][0, 4, 0, 3], x[1][0, 4, 1, 7], x[1][0, 5, 0, 0] = np.inf, -np.inf, np.nan
        kv = [torch.from_numpy(_cache.bf16(a)).to(torch.bfloat16) for a in x]
        width = T // page
        table = g.permutation(B * width + 4)[:B * width].reshape(B, width).astype(np.int32)
        table[2, 2] = -1
        lens, q_lens = [T, 33, 60], [S, 40, 30]
        before = g.integers(0, 256, (B * width + 4, stl.cache4_page_bytes(heads, dim, page)), dtype=np.uint8)
        scales = (0.5, 3.0)
        pages = torch.from_numpy(before).cuda()
        stl.cache4_append(kv[0].cuda(), kv[1].cuda(), pages, dev(table), dev(lens), page, q_lens=dev(q_lens), k_scale=scales[0],
                          v_scale=scales[1])
        want = _cache.Cache4(before.copy(), heads, dim, page)
        back = [np.full((B, S, heads, dim), 9.0) for _ in range(2)]
        for is_v in (0, 1):
            code, sc = _cache.quantise(kv[is_v].double().numpy(), scales[is_v])
            for b in range(B):
                for i in range(q_lens[b]):
                    pos = lens[b] - q_lens[b] + i
                    if pos < 0 or table[b, pos // page] < 0:
                        continue
                    for h in range(heads):
                        want.put(table[b, pos // page], h, pos % page, is_v, code[b, i, h], sc[b, i, h])
                        back[is_v][b, i, h] = want.get(table[b, pos // page], h, pos % page, is_v, scales[is_v])
        assert np.array_equal(pages.cpu().numpy(), want.pages)
        out = tuple(torch.full((B, S, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        got = stl.cache4_read(pages, dev(table), dev(lens), S, heads, dim, page, q_lens=dev(q_lens), k_scale=scales[0],
                              v_scale=scales[1], out=out)
        for is_v in (0, 1):
            assert np.array_equal(got[is_v].double().cpu().numpy(), _cache.bf16(back[is_v].astype(np.float32))), is_v


def test_append_every_quotient():
    """All bf16 numbers of a block's range against each scale mantissa: no tie goes the wrong way."""
    mant = 1 + np.arange(128) / 128
    x = np.concatenate([mant * 2.0 ** e for e in (-3, -2, -1, 0, 1, 2)])
    rows = []
    for top in 6 * (1 + np.arange(8) / 8):
        n = x[x <= top]
        n = np.pad(n, (0, -len(n) % 15))
        for part in n.reshape(-1, 15):
            rows.append(np.concatenate([[top], part * np.where(np.arange(15) % 2, -1, 1)]))
    rows = np.array(rows)
    rows = np.pad(rows, ((0, -len(rows) % 4), (0, 0))).reshape(-1, 64)
    n = len(rows)
    k = torch.from_numpy(rows).to(torch.bfloat16).view(1, n, 1, 64)
    page, width = 16, -(-n // 16)
    for g in (1.0, 0.7, 3.1):
        pages = torch.zeros((width, stl.cache4_page_bytes(1, 64, page)), dtype=torch.uint8, device="cuda")
        table = torch.arange(width, dtype=torch.int32, device="cuda").view(1, width)
        stl.cache4_append(k.cuda(), (-k).cuda(), pages, table, dev([n]), page, k_scale=g, v_scale=g)
        want = _cache.Cache4(np.zeros(pages.shape, np.uint8), 1, 64, page)
        for is_v, sign in ((0, 1), (1, -1)):
            code, sc = _cache.quantise(sign * k.double().numpy()[0, :, 0], g)
            for i in range(n):
                want.put(i // page, 0, i % page, is_v, code[i], sc[i])
        assert np.array_equal(pages.cpu().numpy(), want.pages), g


def test_a_layer_step():
    """A decode step as a layer runs it: the indexer picks entries of a sequence whose compressed rows
    lie in a 4-bit cache, the attention reads them, and the window's result joins it by the lse's."""
    sh = synth.small(2, 1024, 4, 64, 128, 64, seed=3, kc_kind="ar1")
    q, w, kc = _gpu.inputs(sh, seed=3)
    t0 = sh.S - 1
    qd, wd = _gpu.to_dev_bf16(q[:, -1:].copy()), torch.from_numpy(w[:, -1:].copy()).cuda()
    idx, _ = stl.indexer_decode(qd, wd, _gpu.to_dev_bf16(kc), t0, sh.m, sh.topk)
    c = Filled(2, sh.T, 1, 128, 32, seed=5)
    qa = queries(2, 1, 128, 128, seed=6)
    pages, table = c.on_gpu()
    T = dev([sh.T] * 2)
    o1, l1 = stl.cache4_attention(qa, pages, table, T, 1, 32, idx=idx)
    _, k, v = tw.inputs(2, 1, 500, 128, 1, 128, seed=7)
    o2, l2 = stl.window_attention(qa, k, v, 128, 4)
    top = torch.maximum(l1, l2)
    a, b = torch.exp(l1 - top), torch.exp(l2 - top)
    got = ((a[..., None] * o1.float() + b[..., None] * o2.float()) / (a + b)[..., None]).double().cpu().numpy()
    near = idx.cpu().numpy()
    for r in range(2):
        sel = near[r, 0][near[r, 0] >= 0]
        win = np.flatnonzero(_cache.visible(499, 500, 128, 4))
        kk = np.concatenate([c.kv[0].numpy()[r, sel, 0], k.double().cpu().numpy()[r, win, 0]])
        vv = np.concatenate([c.kv[1].numpy()[r, sel, 0], v.double().cpu().numpy()[r, win, 0]])
        for h in range(0, 128, 17):
            o, aw, _, _ = _cache.attend(qa.double().cpu().numpy()[r, 0, h], kk, vv, 128 ** -0.5)
            # two results of 2^-8 each for the probabilities and the rounding, joined in fp32
            assert np.all(np.abs(got[r, 0, h] - o) <= 2.0 ** -7 * aw * 1.01 + 1e-5)


TILE_CASES = [
    # B, S, T, H, Hk, D, page, window, sinks, topk
    (1, 1, 40, 128, 1, 128, 16, 0, 0, 0),      # fewer keys than a block
    (3, 1, 700, 64, 1, 64, 32, 0, 0, 0),       # a cluster joins the chunks
    (2, 1, 1500, 200, 1, 128, 64, 0, 0, 0),    # two row tiles of a query
    (1, 9, 600, 24, 3, 128, 16, 100, 61, 0),   # 72 rows, a window with sinks
    (2, 50, 130, 8, 8, 64, 16, 0, 0, 0),       # a chunk of 50 queries, one head a group
    (2, 2, 500, 128, 1, 128, 64, 0, 0, 300),   # listed entries
]


@pytest.mark.parametrize("B,S,T,H,Hk,D,page,window,sinks,topk", TILE_CASES)
@pytest.mark.parametrize("chunk", [0, 128])
def test_tiles_against_formula(B, S, T, H, Hk, D, page, window, sinks, topk, chunk):
    """33 rows of a kv head and more: the 128-row tiles, with few and with many chunks of a tile's keys."""
    c = Filled(B, T, Hk, D, page, seed=T, k_scale=2.0, v_scale=0.5)
    q = queries(B, S, H, D, seed=T + 1)
    g = np.random.default_rng(T)
    lens = [T] + [int(x) for x in g.integers(0, T, B - 1)]
    q_lens = [S] + [max(1, S - 1)] * (B - 1)
    idx = see = None
    if topk:
        idx = g.integers(-1, T, (B, S, topk)).astype(np.int32)
        see = lambda b, i: np.array([j for j in idx[b, i] if 0 <= j < lens[b]], int)  # noqa: E731
    out, lse = attend(c, q, lens, q_lens, window, sinks, idx=idx, opts=stl.options(key_chunk=chunk) if chunk else None)
    rows = {(b, i) for b in range(B) for i in {0, 1, S // 2, S - 1}}
    check(c, q, window, sinks, lens, q_lens, out, lse, rows=rows, see=see)


def test_tiles_one_cta():
    """A single persistent CTA goes through every item."""
    c = Filled(3, 200, 2, 128, 16, seed=21)
    q = queries(3, 1, 80, 128, seed=22)
    out, lse = attend(c, q, [200, 0, 131], [1, 1, 1], opts=stl.options(grid_ctas=1))
    check(c, q, 0, 0, [200, 0, 131], [1, 1, 1], out, lse)


@pytest.mark.parametrize("H,S", [(8, 1), (8, 4), (24, 1)])
def test_many_ragged_sequences(H, S):
    """Equal shares of the steps of many sequences, most of them short, some without a token."""
    B, T, Hk, D, page = 90, 400, 2, 64, 16
    c = Filled(B, T, Hk, D, page, seed=H)
    q = queries(B, S, H, D, seed=S)
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.choice([0, 1, 5, 33, 64, 399, 400], B)]
    q_lens = [int(x) for x in g.integers(0, S + 1, B)]
    for chunk in (0, 128):
        out, lse = attend(c, q, lens, q_lens, opts=stl.options(key_chunk=chunk) if chunk else None)
        check(c, q, 0, 0, lens, q_lens, out, lse)


def test_same_bits_again():
    c = Filled(5, 900, 2, 128, 32, seed=31)
    lens = [900, 20, 555, 0, 431]
    for H in (8, 80):
        q = queries(5, 1, H, 128, seed=32)
        first = attend(c, q, lens, [1] * 5)
        for _ in range(3):
            again = attend(c, q, lens, [1] * 5)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_two_streams_and_a_graph():
    """Calls that overlap on two streams, and a captured decode step whose lengths grow in place."""
    c = Filled(4, 640, 2, 128, 16, seed=41)
    pages, table = c.on_gpu()
    sets = []
    for H in (8, 80):
        q = queries(4, 1, H, 128, seed=H)
        want = stl.cache4_attention(q, pages, table, dev([640, 100, 333, 1]), 2, 16)
        sets.append((q, want))
    streams = [torch.cuda.Stream() for _ in sets]
    lens = dev([640, 100, 333, 1])
    torch.cuda.synchronize()
    for _ in range(5):
        got = [stl.cache4_attention(q, pages, table, lens, 2, 16, stream=s) for (q, _), s in zip(sets, streams)]
        torch.cuda.synchronize()
        for (_, want), have in zip(sets, got):
            assert torch.equal(want[0], have[0]) and torch.equal(want[1], have[1])
    for q, _ in sets:
        n = dev([639, 99, 332, 1])
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
        stl.cache4_attention(q, pages, table, n, 2, 16, out=out, lse=lse)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            stl.cache4_attention(q, pages, table, n, 2, 16, out=out, lse=lse)
        for lens_now in ([640, 100, 333, 1], [17, 640, 0, 500]):
            n.copy_(dev(lens_now))
            graph.replay()
            want = stl.cache4_attention(q, pages, table, dev(lens_now), 2, 16)
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_pools_beyond_four_gigabytes():
    """Pages whose offsets pass 32 bits: written, read back and attended to like the first ones."""
    heads, dim, page = 8, 128, 64
    n = (5 << 30) // stl.cache4_page_bytes(heads, dim, page)
    pages = torch.zeros((n, stl.cache4_page_bytes(heads, dim, page)), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(50)
    k, v = (torch.randn((1, 100, heads, dim), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    results = []
    for table in ([[3, 1]], [[n - 1, n - 7]]):
        t, lens = dev(table), dev([100])
        stl.cache4_append(k, v, pages, t, lens, page)
        back = stl.cache4_read(pages, t, lens, 100, heads, dim, page)
        att = [stl.cache4_attention(queries(1, 1, H, dim, seed=H), pages, t, lens, heads, page) for H in (16, 320)]
        results.append([*back, *[x for a in att for x in a]])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    refs = torch.zeros(n, dtype=torch.int32, device="cuda")
    refs[[n - 1, n - 7]] = 1
    table, refs2, live = stl.cache_compact(pages, refs, dev([[n - 1, n - 7]]))
    assert live.item() == 2 and table.tolist() == [[1, 0]] and refs2[:2].tolist() == [1, 1]
    assert torch.equal(pages[0], pages[n - 7]) and torch.equal(pages[1], pages[n - 1])


def test_python_refusals():
    c = Filled(2, 64, 2, 64, 16, seed=60)
    pages, table = c.on_gpu()
    lens = dev([64, 64])
    q = queries(2, 1, 8, 64, seed=61)
    ok = dict(qa=q, pages=pages, table=table, lens=lens, heads=2, page=16)
    stl.cache4_attention(**ok)
    for bad in (dict(qa=q.float()), dict(qa=q[0]), dict(qa=q.cpu()), dict(qa=None), dict(qa=torch.stack([q, q], -1)[..., 0]), dict(pages=pages[:, :-16]),
                dict(pages=pages.int()), dict(table=table.long()), dict(table=table[:1]), dict(lens=lens.cpu()), dict(lens=lens[:1]),
                dict(heads=4), dict(page=17), dict(q_lens=lens.float()), dict(idx=table), dict(out=q.float()), dict(lse=q),
                dict(workspace=lens)):
        with pytest.raises(ValueError):
            stl.cache4_attention(**{**ok, **bad})
    for bad in (dict(window=-1), dict(sinks=2), dict(k_scale=0.0), dict(scale=float("nan")), dict(idx=torch.zeros((2, 1, 2049), dtype=torch.int32,
                                                                                                                 device="cuda"))):
        with pytest.raises(stl.StreamIndexError):
            stl.cache4_attention(**{**ok, **bad})
    with pytest.raises(TypeError):
        stl.cache4_attention(**{**ok, "heads": 2.5})
    k = queries(2, 3, 2, 64, seed=62)
    for bad in (dict(v=k[:1]), dict(k=k.half()), dict(table=table[0]), dict(page=3)):
        with pytest.raises(ValueError):
            stl.cache4_append(**{**dict(k=k, v=k, pages=pages, table=table, lens=lens, page=16), **bad})
    with pytest.raises(ValueError):
        stl.cache_fork(pages[:-1], torch.zeros(pages.shape[0], dtype=torch.int32, device="cuda"), table, lens, lens, lens, 16)
    with pytest.raises(ValueError):
        stl.cache_extend(torch.zeros(4, device="cuda"), table, lens, 16)
