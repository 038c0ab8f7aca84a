"""Window attention on the GPU (si_window_attention) against 64-bit rows.

Tolerance, from the arithmetic.  a = sum_j p_j |v_j| is a row's weighted magnitude.  Products of
bf16 are exact in fp32; a dot product of D terms summed in fp32 in any order is off by at most
D 2^-24 sum_d |q_d k_d|, times the scale: e.  A probability is then off by 2 e relative (itself and
the normaliser) plus 2^-20 for the exponential and the rescaling, and by 2^-8 from its rounding to
bf16 (half a step); the sum of up to n values adds n 2^-24, the output's rounding 2^-8 |o|.  So
  |out - o| <= (2^-8 + 2 e + 2^-20 + n 2^-24) a (1 + 2^-8) + 2^-8 |o|
  |lse - l| <= e + 2^-20 + n 2^-24 + 2^-22 |l|."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import streaming_top_lightning_b200 as stl
from tests import _cache

pytestmark = pytest.mark.gpu

U_BF16 = torch.finfo(torch.bfloat16).eps / 2


def inputs(B, S, T, H, Hk, D, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return tuple((torch.randn(s, generator=g) * x).to(torch.bfloat16).cuda()
                 for s, x in (((B, S, H, D), spread), ((B, T, Hk, D), 1.0), ((B, T, Hk, D), 1.0)))


def check(q, k, v, window, sinks, lens, q_lens, out, lse, u=U_BF16, tiny=0.0, scale=None, fill=None,
          rows=None, see=None):
    """Every live row (or those listed) against the formula; the others against ``fill``."""
    B, S, H, D = q.shape
    Hk = k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    qn, kn, vn = (x.double().cpu().numpy() for x in (q, k, v))
    on, ln = out.double().cpu().numpy(), lse.double().cpu().numpy()
    worst = 0.0
    for b in range(B):
        for i in range(S):
            if rows is not None and (b, i) not in rows:
                continue
            if i >= q_lens[b]:
                if fill is not None:
                    assert np.all(on[b, i] == fill) and np.all(ln[b, i] == fill), (b, i)
                continue
            t = lens[b] - q_lens[b] + i
            sel = np.flatnonzero(_cache.visible(t, lens[b], window, sinks))
            if see is not None:
                sel = see(b, i)
            for h in range(H):
                kk, vv = kn[b, sel, h * Hk // H], vn[b, sel, h * Hk // H]
                with np.errstate(invalid="ignore"):
                    o, a, l, big = _cache.attend(qn[b, i, h], kk, vv, scale)
                n = len(sel)
                e = D * 2.0 ** -24 * big * scale
                rel = u + 2 * e + 2.0 ** -20 + n * 2.0 ** -24
                tol = rel * (1 + 2.0 ** -8) * a + U_BF16 * np.abs(o) + tiny * np.abs(vv).sum(0) + 1e-30
                err = np.abs(on[b, i, h] - o)
                assert np.all(np.isfinite(on[b, i, h]) == np.isfinite(o)), (b, i, h)
                assert np.all(err <= tol), (b, i, h, float((err / tol).max()))
                if l == -np.inf:
                    assert ln[b, i, h] == -np.inf, (b, i, h)
                else:
                    assert abs(ln[b, i, h] - l) <= e + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * abs(l), (
                        b, i, h, ln[b, i, h], l)
                worst = max(worst, float((err / tol).max()))
    return worst


def run(q, k, v, window, sinks, lens=None, q_lens=None, **kw):
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    B, S, H, D = q.shape
    out = torch.full((B, S, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, S, H), 7.0, device="cuda")
    r = stl.window_attention(q, k, v, window, sinks, lens=dev(lens), q_lens=dev(q_lens), out=out, lse=lse, **kw)
    assert r[0] is out and r[1] is lse
    torch.cuda.synchronize()
    assert stl.device_error() == 0
    return out, lse


CASES = [
    # B, S, T, H, Hk, D, window, sinks
    (1, 1, 1, 1, 1, 64, 1, 0),           # one token, one key
    (2, 1, 300, 8, 1, 64, 128, 4),       # a decode step
    (3, 1, 1000, 24, 8, 128, 100, 3),    # three heads a group
    (1, 1, 5000, 16, 2, 128, 4096, 4),   # a long window: several CTAs a tile
    (2, 5, 64, 4, 4, 64, 7, 1),          # drafted tokens, one head a group
    (1, 37, 37, 8, 8, 128, 16, 2),       # a whole short prompt
    (2, 130, 200, 6, 2, 64, 33, 0),      # a chunk behind 70 cached tokens
    (1, 3, 90, 128, 1, 128, 40, 5),      # 128 heads on one kv head
    (1, 40, 40, 20, 4, 128, 10 ** 9, 0), # a window longer than anything: causal attention
    (1, 70, 70, 8, 2, 64, 1, 0),         # each token sees itself alone
    (1, 9, 500, 12, 12, 64, 64, 1000),   # more sinks than tokens
]


@pytest.mark.parametrize("B,S,T,H,Hk,D,window,sinks", CASES)
def test_against_formula(B, S, T, H, Hk, D, window, sinks):
    q, k, v = inputs(B, S, T, H, Hk, D, seed=B * S + T)
    out, lse = run(q, k, v, window, sinks)
    check(q, k, v, window, sinks, [T] * B, [S] * B, out, lse)


@pytest.mark.parametrize("S,D,H,Hk", [(1, 128, 8, 2), (7, 64, 6, 3), (50, 128, 4, 1), (300, 64, 16, 4)])
def test_ragged(S, D, H, Hk):
    """Lengths from nothing to everything: rows before the first token see no key, rows past q_lens stay."""
    T = 2 * S + 100
    lens = [T, 0, 1, S // 2, T // 3, T + 50, -3]
    q_lens = [S, S, S, S, S // 2, S + 9, 1]
    q, k, v = inputs(len(lens), S, T, H, Hk, D, seed=S)
    # what lies past a sequence's end is never used
    for b, n in enumerate(lens):
        k[b, max(0, min(n, T)):] = float("nan")
        v[b, max(0, min(n, T)):] = float("inf")
    out, lse = run(q, k, v, 30, 2, lens, q_lens)
    lens = [min(max(n, 0), T) for n in lens]
    q_lens = [min(n, S) for n in q_lens]
    check(torch.nan_to_num(q), torch.nan_to_num(k, nan=0.0), torch.nan_to_num(v, posinf=0.0), 30, 2, lens, q_lens, out, lse,
          fill=7.0)


@pytest.mark.parametrize("S", [1, 6, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3e38])
def test_unseen_keys_do_not_matter(S, bad):
    """Keys outside every window, and keys that only some queries see, hold anything."""
    T, window, sinks = 400, 24, 3
    q, k, v = inputs(1, S, T, 4, 2, 128, seed=5)
    t0 = T - S
    hole = slice(sinks, max(sinks, t0 - window + 1))
    k[:, hole], v[:, hole] = bad, bad
    k[:, T - 1], v[:, T - 1] = bad, bad  # the last token: seen by its own query alone
    out, lse = run(q, k, v, window, sinks)
    kz, vz = k.clone(), v.clone()
    kz[:, hole], vz[:, hole], kz[:, T - 1], vz[:, T - 1] = 0, 0, 0, 0
    check(q, kz, vz, window, sinks, [T], [S], out, lse, rows={(0, i) for i in range(S - 1)})


def test_infinite_values_are_kept():
    """An infinite value that a query sees reaches its output, as in the formula."""
    q, k, v = inputs(1, 2, 50, 4, 4, 64, seed=6)
    v[0, 20, 1, 5] = float("inf")
    out, _ = run(q, k, v, 100, 0)
    assert torch.isposinf(out[0, :, 1, 5]).all()
    out[0, :, 1, 5] = 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("chunk", [128, 256, 1024])
def test_key_chunks(chunk):
    """One row's keys shared by several CTAs."""
    q, k, v = inputs(2, 1, 3000, 8, 2, 128, seed=chunk)
    lens = [3000, 700]
    out, lse = run(q, k, v, 2500, 4, lens, [1, 1], opts=stl.options(key_chunk=chunk))
    check(q, k, v, 2500, 4, lens, [1, 1], out, lse)


def test_peaked_softmax():
    """Logits that spread by hundreds: the running maximum moves and most weights vanish."""
    q, k, v = inputs(1, 40, 300, 4, 2, 64, seed=9, spread=30.0)
    out, lse = run(q, k, v, 200, 4, scale=1.0)
    check(q, k, v, 200, 4, [300], [40], out, lse, scale=1.0)


def test_zero_scale_is_the_mean():
    q, k, v = inputs(1, 1, 100, 2, 1, 64, seed=10)
    out, lse = run(q, k, v, 50, 0, scale=0.0)
    want = v[0, 50:, 0].double().mean(0)
    assert (out[0, 0].double() - want).abs().max() <= 2.0 ** -8 * (want.abs().max() + v[0, 50:].double().abs().mean())
    assert (lse - np.log(50)).abs().max() < 1e-5


def test_same_bits_again():
    q, k, v = inputs(2, 1, 4000, 16, 2, 128, seed=11)
    a = [x.clone() for x in run(q, k, v, 3500, 4)]
    for _ in range(3):
        b = run(q, k, v, 3500, 4)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_and_streams():
    """Captured and replayed on new inputs, and on a stream of its own, with the caller's workspace."""
    B, S, T, H, Hk, D = 2, 1, 3000, 8, 2, 128
    sets = [inputs(B, S, T, H, Hk, D, seed=20 + i) for i in range(3)]
    q, k, v = (x.clone() for x in sets[0])
    lens = torch.tensor([3000, 1234], dtype=torch.int32, device="cuda")
    want = [stl.window_attention(*s, 2000, 4, lens=lens) for s in sets]
    out, lse = stl.window_attention(q, k, v, 2000, 4, lens=lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stl.window_attention(q, k, v, 2000, 4, lens=lens, out=out, lse=lse)
    for s, w in zip(sets, want):
        for x, y in zip((q, k, v), s):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = [stl.window_attention(*s, 2000, 4, lens=lens, stream=other) for s in sets]
    other.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


TILE_CASES = [
    # B, S, T, H, Hk, D, window, sinks
    (1, 64, 64, 1, 1, 128, 64, 0),
    (1, 129, 400, 2, 2, 64, 100, 4),      # one head a group: 128 queries a tile
    (2, 300, 300, 3, 1, 128, 57, 1),      # three heads a group: rows that no query has
    (1, 33, 1000, 128, 1, 128, 300, 200), # one query a tile, two sink blocks
    (1, 500, 777, 12, 4, 64, 128, 0),
    (1, 200, 2000, 8, 1, 128, 1500, 5),
    (1, 70, 70, 100, 1, 64, 10 ** 9, 0),
]


@pytest.mark.parametrize("B,S,T,H,Hk,D,window,sinks", TILE_CASES)
def test_tiles_against_formula(B, S, T, H, Hk, D, window, sinks):
    q, k, v = inputs(B, S, T, H, Hk, D, seed=S + T)
    out, lse = run(q, k, v, window, sinks)
    rows = {(b, i) for b in range(B) for i in {*range(0, S, 7), S - 1, S - 2, 127 % S, 128 % S}}
    check(q, k, v, window, sinks, [T] * B, [S] * B, out, lse, rows=rows)


def test_tiles_zero_scale():
    q, k, v = inputs(1, 80, 80, 2, 1, 64, seed=12)
    out, lse = run(q, k, v, 50, 0, scale=0.0)
    for i in (0, 10, 79):
        seen = v[0, max(0, i - 49):i + 1, 0].double()
        err = (out[0, i].double() - seen.mean(0)).abs()
        assert (err <= 2.0 ** -7 * (seen.abs().mean(0) + 1e-3)).all()
        assert (lse[0, i] - np.log(len(seen))).abs().max() < 1e-5


def test_tiles_agree_with_rows():
    """The two kernels of the window attention on the same call (key chunks fix the rows kernel)."""
    q, k, v = inputs(2, 90, 600, 16, 2, 128, seed=13)
    a = run(q, k, v, 333, 3, [600, 411], [90, 77])
    b = run(q, k, v, 333, 3, [600, 411], [90, 77], opts=stl.options(key_chunk=1024))
    assert (a[0].float() - b[0].float()).abs().max() <= 2.0 ** -6 * v.abs().max()
    assert (a[1] - b[1]).abs().max() <= 1e-4
    check(q, k, v, 333, 3, [600, 411], [90, 77], *b, rows={(0, 0), (0, 89), (1, 40), (1, 76)}, fill=None)


def test_caches_beyond_four_gigabytes():
    """Keys whose offsets pass 32 bits (elements and bytes), by both kernels."""
    T, Hk, D = 600_000, 32, 128
    k = torch.zeros((1, T, Hk, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    n = 512  # the two calls then cut the keys into the same steps
    _, ks, vs = inputs(1, 40, n, 32, Hk, D, seed=70)
    k[:, T - n:], v[:, T - n:] = ks, vs
    for S in (1, 40, 300):
        q = inputs(1, S, n, 32, Hk, D, seed=S)[0]
        a = stl.window_attention(q, k, v, 100, 0)
        b = stl.window_attention(q, ks, vs, 100, 0)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tiles_few_ctas_and_a_graph():
    q, k, v = inputs(2, 200, 300, 8, 2, 128, seed=71)
    lens = torch.tensor([300, 250], dtype=torch.int32, device="cuda")
    want = stl.window_attention(q, k, v, 64, 4, lens=lens)
    got = stl.window_attention(q, k, v, 64, 4, lens=lens, opts=stl.options(grid_ctas=3))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stl.window_attention(q, k, v, 64, 4, lens=lens, out=out, lse=lse)
    for now in ([300, 250], [200, 300], [7, 0]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        want = stl.window_attention(q, k, v, 64, 4, lens=lens)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_python_refusals():
    q, k, v = inputs(1, 2, 50, 4, 2, 64, seed=72)
    for bad in (dict(qa=q.float()), dict(ka=k[0]), dict(va=v[:, :-1]), dict(qa=q.cpu()), dict(ka=k.transpose(1, 2)), dict(lens=q),
                dict(lens=torch.zeros(1, dtype=torch.int32)), dict(q_lens=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(out=q.float()),
                dict(va=None)):
        with pytest.raises(ValueError):
            stl.window_attention(**{**dict(qa=q, ka=k, va=v, window=8), **bad})
    for bad in (dict(window=0), dict(sinks=-1), dict(scale=-2.0), dict(qa=inputs(1, 2, 50, 3, 2, 64, seed=1)[0])):
        with pytest.raises(stl.StreamIndexError):
            stl.window_attention(**{**dict(qa=q, ka=k, va=v, window=8), **bad})
