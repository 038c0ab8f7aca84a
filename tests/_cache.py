"""Plain implementations of the key/value cache operators for their tests: 64-bit numpy and Python
lists, sharing no code with the library."""

from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every non-negative finite E4M3 number by its code (0x7F is NaN)
E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                 for c in range(127)])


def bf16(x):
    """x rounded to bf16 (nearest, ties to even), as float64; NaN and infinities stay."""
    f = np.asarray(x, np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(f), r, f).astype(np.float64)


def nearest(x, numbers):
    """Index of the number nearest to each x >= 0 (numbers ascending from 0), ties to the even index."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(numbers, x), 1, len(numbers) - 1)
    lo = hi - 1
    up, down = numbers[hi] - x, x - numbers[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise(x, g):
    """Rows x [..., D] as (E2M1 codes 0..15 [..., D], E4M3 scale codes [..., D/16])."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    blk = x.reshape(*x.shape[:-1], -1, 16)
    amax = np.abs(blk).max(-1)
    # the library's quotients are fp32: amax / (6 g) and x / (g s), each rounded once
    with np.errstate(over="ignore", invalid="ignore"):
        s = (amax.astype(np.float32) / np.float32(np.float32(6) * np.float32(g))).astype(np.float64)
        sc = nearest(np.minimum(s, 448.0), E4M3)
        gs = (E4M3[sc].astype(np.float32) * np.float32(g)).astype(np.float32)
        q = np.abs(blk).astype(np.float32) / np.where(gs > 0, gs, 1)[..., None]
    code = nearest(np.minimum(q.astype(np.float64), 6.0), E2M1)
    code = np.where(gs[..., None] > 0, code | (np.signbit(blk) << 3), 0)
    return code.reshape(x.shape).astype(np.uint8), sc.astype(np.uint8)


def values(code, sc, g):
    """The numbers that codes and scales stand for."""
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    return v * np.repeat(E4M3[sc], 16, axis=-1) * np.float64(np.float32(g))


class Cache4:
    """Pages of a 4-bit cache as bytes."""

    def __init__(self, pages, heads, dim, page):
        self.pages, self.heads, self.dim, self.page = pages, heads, dim, page
        self.block = page * (dim + dim // 8)

    def _at(self, pg, h, slot, is_v):
        base = h * self.block
        c = base + (self.page * self.dim // 2 if is_v else 0) + slot * self.dim // 2
        s = (base + self.page * self.dim + (self.page * self.dim // 16 if is_v else 0)
             + slot * self.dim // 16)
        return self.pages[pg, c:c + self.dim // 2], self.pages[pg, s:s + self.dim // 16]

    def put(self, pg, h, slot, is_v, code, sc):
        c, s = self._at(pg, h, slot, is_v)
        c[:] = code[0::2] | (code[1::2] << 4)
        s[:] = sc

    def get(self, pg, h, slot, is_v, g):
        c, s = self._at(pg, h, slot, is_v)
        code = np.empty(self.dim, np.uint8)
        code[0::2], code[1::2] = c & 15, c >> 4
        return values(code, s, g)


def visible(t, n, window, sinks):
    """Which of the n keys of a sequence the query at position t sees (window 0: no window)."""
    j = np.arange(n)
    see = j <= t
    if window:
        see &= (j > t - window) | (j < sinks)
    return see


def attend(q, k, v, scale):
    """q [D] over k, v [n, D] in 64 bits: (out, weighted |v|, lse, largest |q||k|)."""
    if len(k) == 0:
        z = np.zeros(v.shape[-1])
        return z, z, -np.inf, 0.0
    x = k @ q * scale
    m = x.max()
    if m == -np.inf:
        z = np.zeros(v.shape[-1])
        return z, z, -np.inf, 0.0
    p = np.exp(x - m)
    tot = p.sum()
    p = p / tot
    return p @ v, p @ np.abs(v), m + np.log(tot), float((np.abs(k) @ np.abs(q)).max())


class Pool:
    """The pages of a pool, call by call, in Python lists."""

    def __init__(self, refs, table, lens, page, content=None):
        self.refs, self.lens = [int(x) for x in refs], [int(x) for x in lens]
        self.table = [[int(x) for x in row] for row in table]
        self.page = page
        self.content = content  # [n_pages, bytes] array, or None

    def _take(self):
        for p, r in enumerate(self.refs):
            if r == 0:
                self.refs[p] = 1
                return p
        return -1

    def extend(self, lens):
        missing = 0
        for row, n in zip(self.table, lens):
            for e in range(min(len(row), max(0, -(-int(n) // self.page)))):
                if row[e] < 0:
                    row[e] = self._take()
                    missing += row[e] < 0
        return missing

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.table):
                for e, p in enumerate(self.table[r]):
                    if 0 <= p < len(self.refs):
                        self.refs[p] = max(0, self.refs[p] - 1)
                    self.table[r][e] = -1
                self.lens[r] = 0

    def fork(self, src, dst):
        table, lens = [list(r) for r in self.table], list(self.lens)
        B, width = len(table), len(table[0])
        missing, taken, made = 0, set(), []
        for s, d in zip(src, dst):
            ok = 0 <= s < B and 0 <= d < B and s != d and d not in taken
            if 0 <= d < B:
                taken.add(d)
            ok = ok and lens[d] == 0 and table[d][0] < 0 and lens[s] >= 0
            if ok:
                full, part = divmod(lens[s], self.page)
                ok = full + (part > 0) <= width
                ok = ok and (part == 0 or 0 <= table[s][full] < len(self.refs))
            if ok and part:
                fresh = self._take()
                ok = fresh >= 0
            if not ok:
                missing += 1
                continue
            made.append((s, d, full, fresh if part else -1))
        for s, d, full, fresh in made:
            for e in range(full):
                p = table[s][e]
                self.table[d][e] = p
                if 0 <= p < len(self.refs):
                    self.refs[p] += 1
            if fresh >= 0:
                self.table[d][full] = fresh
                if self.content is not None:
                    self.content[fresh] = self.content[table[s][full]]
            self.lens[d] = lens[s]
        return missing

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        movers = [p for p in live if p >= n]
        to = {p: p for p in live}
        to.update(zip(movers, holes))
        refs = [0] * len(self.refs)
        for p in live:
            refs[to[p]] = self.refs[p]
        if self.content is not None:
            for a, b in zip(movers, holes):
                self.content[b] = self.content[a]
        self.refs = refs
        self.table = [[p if p < 0 or p >= len(refs) else to.get(p, -1) for p in row]
                      for row in self.table]
        return n
