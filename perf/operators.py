"""Cases that measure the key/value cache operators: attention with a sliding window and sinks, the
4-bit paged cache with its append, read-back and attention, and the life of its pages.

``run`` computes each operator in a plain form of elementary torch operations (``own`` false) or calls
the library (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.

The 4-bit cache: ``pages`` is uint8 [n_pages, page_bytes].  A page holds ``page`` tokens of every kv
head, head after head; one head's block is its K codes [page, D/2], V codes [page, D/2], K scales
[page, D/16] and V scales [page, D/16].  Element d of a row is the low (even d) or high (odd d) nibble
of byte d/2, an E2M1 number; its 16-element block has an E4M3 scale, and K and V have one fp32 scale
each on top.  Token j of sequence b lies in page ``table[b, j // page]``.
"""

from __future__ import annotations

import math

import torch

own = False

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDPOINTS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ---------------------------------------------------------------------------- cases


def listed():
    return [
        # one new token of a short conversation: a call that is all latency
        dict(name="window: one token", op="window", B=1, S=1, T=300, H=8, Hk=1, D=64, window=128, sinks=4, ragged=False),
        # a decode step of a batch of ragged sequences, grouped heads
        dict(name="window: decode batch", op="window", B=32, S=1, T=4096, H=32, Hk=8, D=128, window=1024, sinks=4, ragged=True),
        # the prefill of a long prompt
        dict(name="window: prefill", op="window", B=1, S=8192, T=8192, H=64, Hk=8, D=128, window=1024, sinks=4, ragged=False),
        # a prompt's chunk behind what is cached already, odd sizes, padded rows
        dict(name="window: ragged chunk", op="window", B=3, S=777, T=5001, H=24, Hk=8, D=64, window=500, sinks=3, ragged=True),
        # the decode step of the library's benchmark: 64 sequences of 16,384 entries, the indexer's 2,048 each
        dict(name="cache4: listed entries", op="cache4", B=64, S=1, T=16384, H=128, Hk=1, D=128, page=64, window=0, sinks=0, topk=2048, ragged=False),
        # a decode step over whole ragged sequences
        dict(name="cache4: decode batch", op="cache4", B=32, S=1, T=8192, H=32, Hk=8, D=128, page=64, window=0, sinks=0, topk=0, ragged=True),
        # three drafted tokens of four short sequences, a window with sinks
        dict(name="cache4: drafted tokens", op="cache4", B=4, S=3, T=1000, H=32, Hk=8, D=64, page=16, window=256, sinks=4, topk=0, ragged=True),
        # a decode step writes one token per sequence
        dict(name="append: decode step", op="append", B=64, S=1, T=4096, Hk=8, D=128, page=64, ragged=True),
        # a prefill's chunk goes into the cache
        dict(name="append: prefill chunk", op="append", B=4, S=4096, T=8192, Hk=8, D=128, page=128, ragged=True),
        # a step of a beam search: half the rows end, the others are forked onto them and all grow by a token
        dict(name="turn: beam step", op="turn", B=64, T=4096, Hk=8, D=128, page=64, used=0.6),
        # the cache of a long-running server, compacted: small and large pools
        dict(name="compact: small pool", op="compact", B=16, T=1000, Hk=2, D=64, page=16, used=0.5),
        dict(name="compact: large pool", op="compact", B=128, T=8192, Hk=8, D=128, page=64, used=0.7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["window", "window", "cache4", "cache4", "append", "turn", "compact"])
    H, Hk = rng.choice([(8, 1), (16, 2), (32, 8), (64, 8), (24, 8), (12, 12), (20, 4), (128, 1)])
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "window":
        B = _log_int(rng, 1, 32)
        S = 1 if rng.random() < 0.3 else _log_int(rng, 2, 4096)
        while B * S * H > 150000:
            S = max(1, S // 2)
            B = max(1, B // 2)
        T = _log_int(rng, S, 8192)
        return dict(op=op, B=B, S=S, T=T, H=H, Hk=Hk, D=D, window=_log_int(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 61]), ragged=rng.random() < 0.7)
    if op == "cache4":
        B = _log_int(rng, 1, 64)
        S = 1 if rng.random() < 0.6 else rng.randint(2, 9)
        T = _log_int(rng, 16, 16384)
        while B * T * Hk > 1 << 20:
            B = max(1, B // 2)
            T = max(16, T * 3 // 4)
        kind = rng.choice(["whole", "whole", "window", "listed"])
        return dict(op=op, B=B, S=S, T=T, H=H, Hk=Hk, D=D, page=page, window=_log_int(rng, 1, 4096) if kind == "window" else 0,
                    sinks=rng.choice([0, 4, 61]) if kind == "window" else 0,
                    topk=min(2048, _log_int(rng, 1, T)) if kind == "listed" else 0, ragged=rng.random() < 0.7)
    if op == "append":
        B = _log_int(rng, 1, 64)
        S = 1 if rng.random() < 0.3 else _log_int(rng, 2, 4096)
        while B * S > 16384:
            S = max(1, S // 2)
        return dict(op=op, B=B, S=S, T=S + _log_int(rng, 1, 4096), Hk=Hk, D=D, page=page, ragged=rng.random() < 0.7)
    return dict(op=op, B=_log_int(rng, 2, 128), T=_log_int(rng, page, 4096), Hk=rng.choice([1, 2, 8]), D=D, page=page, used=rng.choice([0.3, 0.5, 0.75]))


# ---------------------------------------------------------------------------- inputs


def _page_bytes(Hk, D, page):
    return Hk * page * (D + D // 8)


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rows(g, shape, spread):
    """bf16 rows of normal numbers, one in fifty of them four times as large."""
    x = torch.randn(shape, generator=g, device="cuda") * spread
    heavy = torch.rand(shape[:-1], generator=g, device="cuda") < 0.02
    return torch.where(heavy[..., None], 4 * x, x).to(torch.bfloat16)


def _lengths(g, c, least):
    """Lengths of the sequences in tokens, and how many of them are this call's."""
    B, S, T = c["B"], c["S"], c["T"]
    if not c["ragged"]:
        return torch.full((B,), T, dtype=torch.int32, device="cuda"), torch.full((B,), S, dtype=torch.int32, device="cuda")
    u, w = torch.rand((2, B), generator=g, device="cuda")
    lens = (least + u * (T - least)).round().to(torch.int32)
    lens[0] = T
    q_lens = torch.minimum((1 + w * (S - 1)).round().to(torch.int32), lens)
    q_lens[0] = min(S, T)
    return lens, q_lens


def _quantise(x, scale):
    """(codes, scales) of the rows of x, as bytes."""
    D = x.shape[-1]
    f = x.float().unflatten(-1, (D // 16, 16))
    s = (f.abs().amax(-1) / (6 * scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = f / (scale * s.float())[..., None]
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, mid in enumerate(MIDPOINTS):  # a tie goes to the even code
        code += (a >= mid) if i % 2 else (a > mid)
    code |= (f < 0).to(torch.uint8) << 3
    code = torch.where((s.float() == 0)[..., None], torch.zeros_like(code), code).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _segments(pages, Hk, D, page):
    """Views of a page tensor's K codes, V codes, K scales and V scales, each [n_pages, Hk, page, bytes]."""
    block = pages.view(pages.shape[0], Hk, page * (D + D // 8))
    at, out = 0, []
    for width in (D // 2, D // 2, D // 16, D // 16):
        out.append(block[:, :, at:at + page * width].unflatten(-1, (page, width)))
        at += page * width
    return out


def _fill(g, pages, Hk, D, page):
    """Random cache contents, some pages at a time."""
    some = max(1, (1 << 26) // (Hk * page * D))
    for first in range(0, pages.shape[0], some):
        part = pages[first:first + some]
        kc, vc, ks, vs = _segments(part, Hk, D, page)
        for c, s in ((kc, ks), (vc, vs)):
            q = _quantise(_rows(g, (part.shape[0], Hk, page, D), 1.0), 1.0)
            c.copy_(q[0])
            s.copy_(q[1])


def prepare(case, seed):
    g = _rng(seed)
    c = dict(case)
    dev = "cuda"
    if c["op"] == "window":
        B, S, T, H, Hk, D = (c[k] for k in ("B", "S", "T", "H", "Hk", "D"))
        lens, q_lens = _lengths(g, c, 1)
        c.update(q=_rows(g, (B, S, H, D), 1.0), k=_rows(g, (B, T, Hk, D), 1.0), v=_rows(g, (B, T, Hk, D), 1.0), lens=lens, q_lens=q_lens,
                 out=torch.zeros((B, S, H, D), dtype=torch.bfloat16, device=dev), lse=torch.zeros((B, S, H), device=dev))
        return c
    B, T, Hk, D, page = (c[k] for k in ("B", "T", "Hk", "D", "page"))
    width = -(-(T + 1) // page)
    size = _page_bytes(Hk, D, page)
    if c["op"] in ("cache4", "append"):
        S = c["S"]
        lens, q_lens = _lengths(g, c, 1)
        n = B * width
        table = torch.randperm(n, generator=g, device=dev).to(torch.int32).view(B, width)
        pages = torch.zeros((n, size), dtype=torch.uint8, device=dev)
        c.update(pages=pages, table=table, lens=lens, q_lens=q_lens, k_scale=0.5, v_scale=2.0)
        if c["op"] == "append":
            c.update(k=_rows(g, (B, S, Hk, D), 1.0), v=_rows(g, (B, S, Hk, D), 1.0),
                     out=tuple(torch.zeros((B, S, Hk, D), dtype=torch.bfloat16, device=dev) for _ in range(2)))
            return c
        _fill(g, pages, Hk, D, page)
        H = c["H"]
        c.update(q=_rows(g, (B, S, H, D), 2.0), idx=None, out=torch.zeros((B, S, H, D), dtype=torch.bfloat16, device=dev),
                 lse=torch.zeros((B, S, H), device=dev))
        if c["topk"]:  # distinct entries of the sequence in a random order, -1 where it has fewer
            order = torch.rand((B, S, T), generator=g, device=dev).topk(c["topk"], dim=-1).indices.to(torch.int32)
            c["idx"] = torch.where(order < lens[:, None, None], order, torch.full_like(order, -1)).contiguous()
        return c
    # a pool in use: sequences of random lengths, their pages anywhere in it
    n = max(8, int(B * width / c["used"]))
    pages = torch.randint(0, 256, (n, size), generator=g, device=dev, dtype=torch.uint8)
    lens = (1 + torch.rand((B,), generator=g, device=dev) * (T - 1)).round().to(torch.int32)
    held = torch.arange(width, device=dev)[None] < -(-lens // page)[:, None]
    table = torch.randperm(n, generator=g, device=dev)[: B * width].to(torch.int32).view(B, width)
    table = torch.where(held, table, torch.full_like(table, -1)).contiguous()
    refs = torch.zeros((n + 1,), dtype=torch.int32, device=dev)
    refs[torch.where(held, table, torch.full_like(table, n)).flatten().long()] = 1
    c.update(pages=pages, lens=lens, table=table, refs=refs[:n].clone())
    if c["op"] == "turn":
        half = B // 2
        rows = torch.randperm(B, generator=g, device=dev).to(torch.int32)
        parents = rows[half:][torch.randint(0, B - half, (half,), generator=g, device=dev)]
        c.update(dst=rows[:half].contiguous(), src=parents.contiguous())
    return c


# ---------------------------------------------------------------------------- plain forms


def _attend(q, k, v, visible, scale):
    """Softmax attention in fp32: q [B,S,H,D], k, v [B,T,Hk,D] or a list of their own for each query [B,S,T,Hk,D];
    visible [B,S,T].  Returns out [B,S,H,D] and lse [B,S,H]."""
    B, S, H, D = q.shape
    if k.dim() == 5:
        q, k, v, visible = (x.flatten(0, 1) for x in (q[:, :, None], k, v, visible[:, :, None]))
    Hk = k.shape[2]
    G = H // Hk
    n, s_q = q.shape[:2]
    qg = q.float().view(n, s_q, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(n, Hk, s_q * G, D)
    kt = k.float().permute(0, 2, 3, 1)
    s = torch.matmul(qg, kt).mul_(scale).view(n, Hk, s_q, G, -1)
    s.masked_fill_(~visible[:, None, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, Hk, s_q * G, -1), v.float().permute(0, 2, 1, 3)).view(n, Hk, s_q, G, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)
    return o.permute(0, 2, 1, 3, 4).reshape(B, S, H, D), lse.permute(0, 2, 1, 3).reshape(B, S, H)


def _visible(lens, q_lens, S, T, window, sinks):
    t = (lens - q_lens)[:, None] + torch.arange(S, device=lens.device)
    j = torch.arange(T, device=lens.device)
    see = (j <= t[..., None]) & (j < lens[:, None, None])
    return see & ((j > t[..., None] - window) | (j < sinks)) if window else see


def _kept(st, o, lse):
    """The outputs with the rows that no query has left as they were."""
    live = torch.arange(st["S"], device=o.device)[None] < st["q_lens"][:, None]
    return torch.where(live[..., None, None], o.to(torch.bfloat16), st["out"]), torch.where(live[..., None], lse, st["lse"])


def _values(codes, scales, scale):
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() * scale
    return table[nib.int()] * s.repeat_interleave(16, -1)


def _cached(st, pos, b):
    """K and V of the tokens at positions pos of the sequences b, in fp32 [..., Hk, D]."""
    Hk, D, page = st["Hk"], st["D"], st["page"]
    pg = st["table"][b, pos // page].long()
    kc, vc, ks, vs = (x[pg, :, pos % page] for x in _segments(st["pages"], Hk, D, page))
    return _values(kc, ks, st["k_scale"]), _values(vc, vs, st["v_scale"])


def _new_rows(st):
    """Positions of the call's rows, their sequences, and which of them there are."""
    dev = st["lens"].device
    i = torch.arange(st["S"], device=dev)[None]
    pos = (st["lens"] - st["q_lens"])[:, None] + i
    live = (i < st["q_lens"][:, None]) & (pos >= 0)
    return pos.long(), torch.arange(st["B"], device=dev)[:, None].expand_as(pos), live


def _plain_append(st):
    pos, b, live = _new_rows(st)
    pos, b = pos[live], b[live]
    pg = st["table"][b, pos // st["page"]].long()
    kc, vc, ks, vs = _segments(st["pages"], st["Hk"], st["D"], st["page"])
    for x, c, s, scale in ((st["k"], kc, ks, st["k_scale"]), (st["v"], vc, vs, st["v_scale"])):
        c[pg, :, pos % st["page"]], s[pg, :, pos % st["page"]] = _quantise(x[live], scale)
    k, v = _cached(st, pos, b)
    for out, x in zip(st["out"], (k, v)):
        out[live] = x.to(torch.bfloat16)
    return st["out"]


def _free_list(refs):
    """The free pages in ascending order (then n, the number of pages), and how many there are."""
    n = refs.numel()
    free = refs == 0
    at = torch.where(free, torch.cumsum(free, 0) - 1, torch.full_like(refs, n).long())
    order = torch.full((n + 1,), n, dtype=torch.int64, device=refs.device)
    order[at] = torch.where(free, torch.arange(n, device=refs.device), n)
    order[n] = n
    return order, free.sum()


def _plain_turn(st):
    pages, refs, table, lens = st["pages"], st["refs"], st["table"], st["lens"]
    src, dst, page = st["src"].long(), st["dst"].long(), st["page"]
    n, width = pages.shape[0], table.shape[1]
    col = torch.arange(width, device=table.device)
    # the rows that end
    old = table[dst].flatten().long()
    refs -= torch.zeros((n + 1,), dtype=torch.int32, device=refs.device).index_add_(0, torch.where(old < 0, n, old), torch.ones_like(old, dtype=torch.int32))[:n]
    table[dst] = -1
    lens[dst] = 0
    # the forks: whole pages are shared, a partly filled last one is copied to the lowest free page
    full, part = (lens[src] // page).long(), lens[src] % page > 0
    order, n_free = _free_list(refs)
    rank = torch.cumsum(part, 0) - 1
    made = ~part | (rank < n_free)
    fresh = torch.where(part & made, order[rank.clamp(0, n)], n)
    rows = table[src].long()
    last = rows.gather(1, full.clamp(max=width - 1)[:, None]).squeeze(1)
    copied = part & made
    pages[fresh[copied]] = pages[last[copied]]
    child = torch.where(col < full[:, None], rows, torch.where((col == full[:, None]) & copied[:, None], fresh[:, None], -1))
    child = torch.where(made[:, None], child, -1)
    table[dst] = child.to(torch.int32)
    lens[dst] = torch.where(made, lens[src], 0)
    flat = child.flatten()
    refs += torch.zeros((n + 1,), dtype=torch.int32, device=refs.device).index_add_(0, torch.where(flat < 0, n, flat), torch.ones_like(flat, dtype=torch.int32))[:n]
    lost = (~made).sum()
    # pages for one more token of every row
    need = -(-(lens + 1) // page)
    want = (col[None] < need[:, None]) & (table < 0)
    order, n_free = _free_list(refs)
    rank = torch.cumsum(want.flatten(), 0).view_as(want) - 1
    got = want & (rank < n_free)
    page_of = order[rank.clamp(0, n)]
    table.copy_(torch.where(got, page_of, table.long()))
    refs += torch.zeros((n + 1,), dtype=torch.int32, device=refs.device).index_add_(0, torch.where(got, page_of, n).flatten(), torch.ones((got.numel(),), dtype=torch.int32, device=refs.device))[:n]
    return pages, refs, table, lens, lost.to(torch.int32).view(1), (want & ~got).sum().to(torch.int32).view(1)


def _plain_compact(st):
    pages, refs, table = st["pages"], st["refs"], st["table"]
    n = refs.numel()
    at = torch.arange(n, device=refs.device)
    live = refs > 0
    count = live.sum()
    hole, mover = (~live) & (at < count), live & (at >= count)
    holes, movers = hole.nonzero().squeeze(1), mover.nonzero().squeeze(1)
    pages[holes] = pages[movers]
    to = torch.where(live, at, -1)
    to[movers] = holes
    moved = torch.where(live & ~mover, refs, 0)
    moved[holes] = refs[movers]
    return torch.where(table < 0, table, to[table.long().clamp(min=0)].to(torch.int32)), moved, count.to(torch.int32).view(1), pages


def run(state):
    st = state
    op = st["op"]
    if own:
        import streaming_top_lightning_b200 as stl

        if op == "window":
            return stl.window_attention(st["q"], st["k"], st["v"], st["window"], st["sinks"], lens=st["lens"], q_lens=st["q_lens"], out=st["out"], lse=st["lse"])
        if op == "cache4":
            return stl.cache4_attention(st["q"], st["pages"], st["table"], st["lens"], st["Hk"], st["page"], st["window"], st["sinks"], q_lens=st["q_lens"],
                                        idx=st["idx"], k_scale=st["k_scale"], v_scale=st["v_scale"], out=st["out"], lse=st["lse"])
        if op == "append":
            stl.cache4_append(st["k"], st["v"], st["pages"], st["table"], st["lens"], st["page"], q_lens=st["q_lens"], k_scale=st["k_scale"], v_scale=st["v_scale"])
            return stl.cache4_read(st["pages"], st["table"], st["lens"], st["S"], st["Hk"], st["D"], st["page"], q_lens=st["q_lens"], k_scale=st["k_scale"],
                                   v_scale=st["v_scale"], out=st["out"])
        if op == "turn":
            stl.cache_free(st["refs"], st["table"], st["lens"], st["dst"])
            lost = stl.cache_fork(st["pages"], st["refs"], st["table"], st["lens"], st["src"], st["dst"], st["page"])
            short = stl.cache_extend(st["refs"], st["table"], st["lens"] + 1, st["page"])
            return st["pages"], st["refs"], st["table"], st["lens"], lost, short
        table, refs, live = stl.cache_compact(st["pages"], st["refs"], st["table"])
        return table, refs, live, st["pages"]
    if op == "window":
        see = _visible(st["lens"], st["q_lens"], st["S"], st["T"], st["window"], st["sinks"])
        return _kept(st, *_attend(st["q"], st["k"], st["v"], see, st["D"] ** -0.5))
    if op == "cache4":
        dev = st["lens"].device
        b = torch.arange(st["B"], device=dev)
        if st["idx"] is None:
            j = torch.arange(st["T"], device=dev)
            k, v = _cached(st, j[None].expand(st["B"], -1), b[:, None])
            see = _visible(st["lens"], st["q_lens"], st["S"], st["T"], st["window"], st["sinks"])
        else:
            see = (st["idx"] >= 0) & (st["idx"] < st["lens"][:, None, None])
            k, v = _cached(st, torch.where(see, st["idx"], 0).long(), b[:, None, None])
        return _kept(st, *_attend(st["q"], k, v, see, st["D"] ** -0.5))
    return {"append": _plain_append, "turn": _plain_turn, "compact": _plain_compact}[op](st)


# ---------------------------------------------------------------------------- work


def _pairs(c):
    """(query, key) pairs that see one another and the cache rows that some query sees, from the case alone (ragged
    sequences count with their mean length)."""
    lens = [c["T"]] + [0.5 * (1 + c["T"]) if c["ragged"] else c["T"]] * (c["B"] - 1)
    pairs = rows = 0.0
    for n in lens:
        s = min(n, c["S"] if not c["ragged"] or n == c["T"] else 0.5 * (1 + c["S"]))
        if c.get("topk"):
            k = c["topk"] * n / c["T"]
            pairs, rows = pairs + s * k, rows + min(s * k, n)
            continue
        w = min(c["window"], n) if c["window"] else n
        first = max(0.0, w - (n - s))  # rows whose window still reaches position 0
        in_window = s * w - 0.5 * first * (first - 1) if first > 0 else s * w
        beyond = max(0.0, n - w - s)  # tokens before the first row's window
        pairs += in_window + s * min(c["sinks"], beyond)
        rows += min(n, w + s - 1 + min(c["sinks"], beyond))
    return pairs, rows


def work(case):
    c = case
    if c["op"] in ("window", "cache4"):
        pairs, rows = _pairs(c)
        q = sum([c["S"]] + [(0.5 * (1 + c["S"]) if c["ragged"] else c["S"])] * (c["B"] - 1))
        per_row = 2 * c["Hk"] * (c["D"] * 2 if c["op"] == "window" else c["D"] // 2 + c["D"] // 16)
        return {"bytes": rows * per_row + q * c["H"] * (4 * c["D"] + 4) + (4 * q * c["topk"] if c.get("topk") else 0), "flops": 4.0 * c["D"] * c["H"] * pairs}
    if c["op"] == "append":
        n = sum([c["S"]] + [(0.5 * (1 + c["S"]) if c["ragged"] else c["S"])] * (c["B"] - 1)) * c["Hk"] * 2
        return {"bytes": n * (4 * c["D"] + 2 * (c["D"] // 2 + c["D"] // 16)), "flops": 4.0 * n * c["D"]}
    width = -(-(c["T"] + 1) // c["page"])
    n = max(8, int(c["B"] * width / c["used"]))
    size = _page_bytes(c["Hk"], c["D"], c["page"])
    held = c["B"] * (0.5 * c["T"] / c["page"] + 0.5)
    if c["op"] == "turn":  # a copied page for each child, the children's rows, the counts
        half = c["B"] // 2
        return {"bytes": 2.0 * half * size * (c["page"] - 1) / c["page"] + 4 * (3 * held + n), "flops": float(held)}
    moved = held * (1 - held / n)
    return {"bytes": 2 * moved * size + 4 * (2 * n + 2 * c["B"] * width), "flops": float(n)}


# ---------------------------------------------------------------------------- 64 bits


def _exact_values(codes, scales, scale):
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    e, m = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    sign = 1 - 2 * (nib >> 3).double()
    se, sm = (scales.long() >> 3) & 15, (scales.long() & 7).double() / 8
    s = torch.where(se == 0, sm * 2.0 ** -6, (1 + sm) * torch.exp2(se.double() - 7))
    return sign * mag * s.repeat_interleave(16, -1) * scale


def _exact_rounded(x, scale):
    """What the cache holds of the rows x: each block's scale and each element rounded to the nearest number of their
    formats, found among all of them, ties to the one with the even code."""
    f = x.double().unflatten(-1, (x.shape[-1] // 16, 16))

    def nearest(y, numbers):
        n = torch.tensor(numbers, dtype=torch.float64, device=y.device)
        hi = torch.searchsorted(n, y.contiguous()).clamp(max=len(numbers) - 1)
        lo = (hi - 1).clamp(min=0)
        up, down = n[hi] - y, y - n[lo]
        return n[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]

    e4m3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]
    s = nearest((f.abs().amax(-1) / (6 * scale)).clamp(max=448.0), e4m3) * scale
    y = torch.where(s[..., None] > 0, f.abs() / s[..., None].clamp(min=1e-300), torch.zeros_like(f))
    return (torch.sign(f) * nearest(y.clamp(max=6.0), list(MAGNITUDES)) * s[..., None]).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op in ("turn", "compact"):
        return None
    B, S, Hk, D = st["B"], st["S"], st["Hk"], st["D"]
    lens, q_lens = st["lens"].tolist(), st["q_lens"].tolist()
    if op == "append":
        outs = []
        for x, scale in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
            o = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
            for b in range(B):
                o[b, : q_lens[b]] = _exact_rounded(x[b, : q_lens[b]], scale)
            outs.append(o)
        return tuple(outs)
    H = st["H"]
    G = H // Hk
    out = st["out"].double()
    lse = st["lse"].double()
    for b in range(B):
        n, s = lens[b], q_lens[b]
        j = torch.arange(n, device=out.device)
        if op == "window":
            k, v = st["k"][b, :n].double(), st["v"][b, :n].double()
        else:
            pg, slot = st["table"][b].long()[j // st["page"]], j % st["page"]
            kc, vc, ks, vs = (x[pg, :, slot] for x in _segments(st["pages"], Hk, D, st["page"]))
            k, v = _exact_values(kc, ks, st["k_scale"]), _exact_values(vc, vs, st["v_scale"])
        t = n - s + torch.arange(s, device=out.device)
        if op == "cache4" and st["idx"] is not None:
            weight = torch.zeros((s, n + 1), dtype=torch.float64, device=out.device)  # how often a row lists an entry
            e = st["idx"][b, :s].long()
            weight.scatter_add_(1, torch.where((e < 0) | (e >= n), n, e), torch.ones(e.shape, dtype=torch.float64, device=out.device))
            weight = weight[:, :n]
        else:
            see = j[None] <= t[:, None]
            if st["window"]:
                see &= (j[None] > t[:, None] - st["window"]) | (j[None] < st["sinks"])
            weight = see.double()
        for h in range(Hk):
            q = st["q"][b, :s, h * G:(h + 1) * G].double()
            logit = torch.einsum("sgd,jd->sgj", q, k[:, h]) / math.sqrt(D)
            logit = torch.where(weight[:, None] > 0, logit + torch.log(weight[:, None]), torch.full_like(logit, -math.inf))
            total = torch.logsumexp(logit, -1)
            p = torch.where(torch.isinf(total)[..., None], torch.zeros_like(logit), torch.exp(logit - total[..., None]))
            out[b, :s, h * G:(h + 1) * G] = torch.einsum("sgj,jd->sgd", p, v[:, h])
            lse[b, :s, h * G:(h + 1) * G] = total
    return out, lse
