"""Window attention whose 128-row tiles share their keys in chunks: few query rows that see many keys.

Tolerance: as in test_gpu_window.py, but for the weights.  Within a chunk they are divided by the sum
of the weights as rounded, so the chunk's mean is off by at most 2^-8 (a + |mean|) <= 2^-7 a, a its
mean of |v|; the chunks' means are averaged with weights that are not rounded, so the whole is off by
2^-7 of its own a at most."""

from __future__ import annotations

import pytest
import torch

import streaming_top_lightning_b200 as stl
from tests.test_gpu_window import U_BF16, check, inputs, run

pytestmark = pytest.mark.gpu

U = 2 * U_BF16

CASES = [
    # B, S, T, H, Hk, D, window, sinks
    (1, 40, 4000, 8, 2, 64, 10 ** 9, 0),
    (1, 33, 5003, 6, 1, 128, 3001, 200),    # chunks that end inside the sinks and the window
    (1, 20, 5003, 3, 3, 64, 2050, 2500),    # as many sinks as window keys, one head a group
    (2, 300, 2900, 4, 4, 128, 2500, 130),   # two tiles a pair, several pairs
    (1, 17, 2500, 1, 1, 128, 2499, 1),      # the fewest rows
    (1, 18, 3000, 100, 1, 64, 2900, 0),     # one query a tile
    (3, 5, 2600, 128, 1, 128, 2200, 77),
]


@pytest.mark.parametrize("B,S,T,H,Hk,D,window,sinks", CASES)
def test_against_formula(B, S, T, H, Hk, D, window, sinks):
    q, k, v = inputs(B, S, T, H, Hk, D, seed=S + T)
    out, lse = run(q, k, v, window, sinks)
    rows = {(b, i) for b in range(B) for i in {0, S - 1, S - 2, S // 2, 63 % S, 127 % S, 128 % S}}
    check(q, k, v, window, sinks, [T] * B, [S] * B, out, lse, u=U, rows=rows)


@pytest.mark.parametrize("D", [64, 128])
def test_ragged(D):
    """Sequences of fewer pieces than the longest, of none, and rows that stay as they were."""
    S, T = 50, 4100
    lens = [T, 0, 1, 30, 64, 65, 700, 1999, T + 50]
    q_lens = [S, S, 1, S, 17, S, 33, 1, S + 1]
    q, k, v = inputs(len(lens), S, T, 4, 2, D, seed=D)
    for b, n in enumerate(lens):
        k[b, min(n, T):] = float("nan")
        v[b, min(n, T):] = float("inf")
    out, lse = run(q, k, v, 3000, 70, lens, q_lens)
    q_lens = [min(n, S) for n in q_lens]
    lens = [min(n, T) for n in lens]
    rows = {(b, i) for b in range(len(lens)) for i in (0, 16, 17, 32, 33, 48, 49)}
    check(q, torch.nan_to_num(k, nan=0.0), torch.nan_to_num(v, posinf=0.0), 3000, 70, lens, q_lens, out, lse, u=U, rows=rows,
          fill=7.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3e38])
def test_unseen_keys_do_not_matter(bad):
    S, T, window, sinks = 40, 4000, 3000, 70
    q, k, v = inputs(1, S, T, 4, 2, 128, seed=5)
    hole = slice(sinks, T - S - window + 1)
    k[:, hole], v[:, hole] = bad, bad
    for t in (T - 1, T - 20):  # seen by the queries from their own on
        k[:, t], v[:, t] = bad, bad
    out, lse = run(q, k, v, window, sinks)
    kz, vz = k.clone(), v.clone()
    for t in (hole, T - 1, T - 20):
        kz[:, t], vz[:, t] = 0, 0
    check(q, kz, vz, window, sinks, [T], [S], out, lse, u=U, rows={(0, i) for i in range(20)})


def test_bad_values_that_are_seen():
    """An infinity or NaN that a query sees reaches its output and nothing else."""
    S, T = 30, 4000
    q, k, v = inputs(1, S, T, 2, 1, 64, seed=6)
    v[0, 100, 0, 5] = float("inf")
    v[0, 3000, 0, 9] = float("nan")
    out, lse = run(q, k, v, T, 0)
    assert torch.isposinf(out[..., 5]).all() and torch.isnan(out[..., 9]).all() and torch.isfinite(lse).all()
    out[..., 5], out[..., 9] = 0, 0
    assert torch.isfinite(out).all()
    k[0, 3999, 0, 3] = float("nan")  # the last query alone
    out, lse = run(q, k, v, T, 0)
    assert torch.isnan(out[0, -1]).all() and torch.isnan(lse[0, -1]).all() and torch.isfinite(lse[0, :-1]).all()


@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_spread_of_the_logits(spread):
    """Equal weights, and chunks whose weights all vanish beside another's."""
    q, k, v = inputs(1, 20, 4000, 4, 2, 64, seed=9, spread=spread)
    out, lse = run(q, k, v, 3500, 4, scale=1.0)
    check(q, k, v, 3500, 4, [4000], [20], out, lse, u=U, scale=1.0)


def test_agrees_with_fewer_ctas_and_the_rows_kernel():
    q, k, v = inputs(2, 30, 3000, 16, 2, 128, seed=13)
    a = run(q, k, v, 2800, 3, [3000, 2411], [30, 21])
    b = run(q, k, v, 2800, 3, [3000, 2411], [30, 21], opts=stl.options(grid_ctas=3))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = run(q, k, v, 2800, 3, [3000, 2411], [30, 21], opts=stl.options(key_chunk=1024))
    check(q, k, v, 2800, 3, [3000, 2411], [30, 21], *c, rows={(0, 0), (1, 20)})
    assert (a[1] - c[1]).abs().max() <= 1e-4


def test_graphs_and_streams():
    """Two graphs of the same call with a workspace each, replayed on two streams at once."""
    sets = [inputs(1, 40, 4000, 8, 2, 128, seed=20 + i) for i in range(2)]
    want = [stl.window_attention(*s, 3000, 4) for s in sets]
    calls = []
    for s in sets:
        out, lse = torch.zeros_like(s[0]), torch.zeros(s[0].shape[:3], device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            stl.window_attention(*s, 3000, 4, out=out, lse=lse)
        calls.append((graph, out, lse, torch.cuda.Stream()))
    for _ in range(5):
        for graph, out, lse, stream in calls:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for (_, out, lse, _), w in zip(calls, want):
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_workspace_refusals():
    q, k, v = inputs(1, 40, 4000, 8, 2, 64, seed=30)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(stl.StreamIndexError):
        stl.window_attention(q, k, v, 3000, 4, workspace=small)


@pytest.mark.parametrize("S,T", [(20, 40), (70, 3000)])
@pytest.mark.parametrize("B", [2, 6, 255, 256, 257])
def test_sequences_without_rows(B, S, T):
    """Rows of some sequences only, on both sides of the number of sequences that a CTA lists."""
    if B > 6 and T > 1000:
        T = 200
    g = torch.Generator().manual_seed(B)
    q_lens = torch.randint(0, S + 1, (B,), generator=g)
    q_lens[torch.rand((B,), generator=g) < 0.5] = 0
    lens = (q_lens + torch.randint(0, T - S + 1, (B,), generator=g)).tolist()
    q_lens = q_lens.tolist()
    q, k, v = inputs(B, S, T, 4, 2, 64, seed=B)
    out, lse = run(q, k, v, T - 10, 3, lens, q_lens)
    some = {0, 1, 2, B // 2, B - 3, B - 2, B - 1}
    rows = {(b, i) for b in some for i in (0, 1, S // 2, S - 1)}
    check(q, k, v, T - 10, 3, lens, q_lens, out, lse, u=U, rows=rows, fill=7.0)
    # the rows that no query has, all of them
    dead = torch.arange(S)[None] >= torch.tensor(q_lens)[:, None]
    assert bool((out.cpu()[dead] == 7).all()) and bool((lse.cpu()[dead] == 7).all())
    assert bool((lse.cpu()[~dead] != 7).all())


def test_no_rows_at_all():
    q, k, v = inputs(3, 40, 50, 4, 2, 128, seed=3)
    out, lse = run(q, k, v, 20, 0, [50, 7, 0], [0, 0, 0])
    assert bool((out == 7).all()) and bool((lse == 7).all())
