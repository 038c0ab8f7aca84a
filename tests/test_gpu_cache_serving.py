"""The cache calls together, as a server makes them: prompts, forks, decode steps with drafted tokens,
ends and a compaction, the attention checked against 64 bits after every step.  Tolerances:
test_gpu_cache4.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import streaming_top_lightning_b200 as stl
from tests import _cache
from tests import test_gpu_cache4 as tc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hk,D,page", [(8, 2, 64, 16), (24, 1, 128, 32)])
def test_a_run(H, Hk, D, page):
    B, cap, n = 6, 160, 60
    g = np.random.default_rng(D)
    gs = (0.5, 2.0)
    pages = torch.full((n, stl.cache4_page_bytes(Hk, D, page)), 0x7F, dtype=torch.uint8, device="cuda")  # NaN scales
    refs = torch.zeros(n, dtype=torch.int32, device="cuda")
    table = torch.full((B, cap // page), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kv = [np.zeros((B, cap, Hk, D)) for _ in range(2)]  # what the cache holds

    def grow(new):
        """Append new[b] tokens to each sequence and attend with their queries."""
        S = max(new)
        lens.add_(tc.dev(new))
        now = lens.cpu().numpy()
        assert int(stl.cache_extend(refs, table, lens, page)) == 0
        rows = []
        for is_v in (0, 1):
            x = _cache.bf16(g.standard_normal((B, S, Hk, D)))
            code, sc = _cache.quantise(x, gs[is_v])
            held = _cache.values(code, sc, gs[is_v])
            for b in range(B):
                kv[is_v][b, now[b] - new[b]:now[b]] = held[b, :new[b]]
            rows.append(torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda())
        stl.cache4_append(*rows, pages, table, lens, page, q_lens=tc.dev(new), k_scale=gs[0], v_scale=gs[1])
        q = tc.queries(B, S, H, D, seed=int(now.sum()))
        return look(q, new), q

    def look(q, new):
        out = torch.full_like(q, 7.0)
        lse = torch.full(q.shape[:3], 7.0, device="cuda")
        stl.cache4_attention(q, pages, table, lens, Hk, page, q_lens=tc.dev(new), k_scale=gs[0], v_scale=gs[1], out=out, lse=lse)
        now = lens.cpu().tolist()
        torch.cuda.synchronize()
        assert stl.device_error() == 0
        tc.tw.check(q, torch.from_numpy(kv[0]), torch.from_numpy(kv[1]), 0, 0, now, new, out, lse, u=tc.U_FP16, tiny=2.0 ** -35,
                    fill=7.0)
        return out, lse

    grow([37, 5, 0, page, 0, 0])
    grow([1, 1, 0, 1, 0, 0])
    assert int(stl.cache_fork(pages, refs, table, lens, tc.dev([0, 0, 3]), tc.dev([2, 4, 5]), page)) == 0
    for is_v in (0, 1):
        for s, d in ((0, 2), (0, 4), (3, 5)):
            kv[is_v][d] = kv[is_v][s]
    for i in range(6):
        grow([[1, 1, 1, 1, 1, 1], [3, 1, 2, 3, 0, 1]][i % 2])
    stl.cache_free(refs, table, lens, tc.dev([0, 3]))
    new = [0, 1, 1, 0, 1, 1]
    (out, lse), q = grow(new)
    before = (refs > 0).sum()
    live = stl.cache_compact(pages, refs, table, out=(table, refs))[2]
    assert int(live) == int(before) and bool((refs[:int(live)] > 0).all()) and not bool(refs[int(live):].any())
    again = look(q, new)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    grow([2, 2, 2, 2, 2, 2])  # the emptied rows begin anew
    stl.cache_free(refs, table, lens, tc.dev(list(range(B))))
    assert not bool(refs.any()) and bool((table == -1).all())
