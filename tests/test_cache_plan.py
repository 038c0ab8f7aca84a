"""The plans of the attention calls over a key/value cache, as far as their workspaces show them, and
that a call asks for the workspace that its size query names.  On the host: every call here fails
before it looks for a device."""

import ctypes

import pytest

from streaming_top_lightning_b200 import _lib, build

FAKE = ctypes.c_void_p(4096)  # aligned, never read
ODD = ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def window_size(lib, B, S, T, H, Hk, d, window, sinks=0, opt=None):
    n = ctypes.c_size_t(0)
    assert lib.si_window_attention_workspace_size(B, S, T, H, Hk, d, window, sinks, opt, ctypes.byref(n)) == 0
    return n.value


def cache4_size(lib, width, page, topk, B, S, H, Hk, d, window=0, sinks=0, opt=None):
    n = ctypes.c_size_t(0)
    assert lib.si_cache4_attention_workspace_size(width, page, topk, B, S, H, Hk, d, window, sinks, opt, ctypes.byref(n)) == 0
    return n.value


def pieces(n, rows, d, extra):
    """Partial results of each row that a workspace of n bytes holds: d + 2 numbers each, in three
    arrays that are multiples of 256 bytes."""
    return (n - extra) // (rows * (4 * d + 8))


@pytest.mark.parametrize("B,H,Hk", [(2, 16, 8), (4, 32, 8), (7, 64, 8), (16, 12, 3)])
def test_one_wave_of_ctas(lib, B, H, Hk):
    """Rows of 64 and of 128 bf16 elements: both kernels' rings take 96 KB, so two CTAs an SM hold
    either, and the shares of one wave cut a long sequence into as many pieces."""
    T = 1 << 17
    tiles, rows = B * Hk, B * H
    room = 2 * 148
    most = min(96, max(8, 8 * room // tiles))  # eight times a tile's even part of the wave
    got = []
    for d in (64, 128):
        n = window_size(lib, B, 1, T, H, Hk, d, T)
        assert n > 0
        got.append(pieces(n, rows, d, 8 * (tiles + 1)))
        assert got[-1] <= most, (d, got[-1], most)
    assert got[0] == got[1]


@pytest.mark.parametrize("d", [64, 128])
def test_long_windows_are_shared(lib, d):
    """A window that may be longer than most sequences does not tie a call to its longest one."""
    T = 1 << 16
    assert window_size(lib, 37, 1, T, 32, 8, d, T) > 0
    assert window_size(lib, 37, 1, T, 32, 8, d, 512) == 0  # a CTA a tile: all see as much
    assert cache4_size(lib, T // 64, 64, 0, 74, 1, 32, 8, d, T) > 0
    assert cache4_size(lib, T // 64, 64, 0, 74, 1, 32, 8, d, 512) == 0


WINDOWS = [(B, S, T, H, Hk, d, w, n, chunk) for B in (1, 5, 64, 700) for S, T in ((1, 30), (1, 40000), (3, 5000), (40, 9000), (600, 60000))
           for H, Hk, d in ((1, 1, 64), (8, 2, 128), (24, 8, 64), (128, 1, 128)) for w, n in ((1, 0), (300, 4), (10 ** 9, 0)) for chunk in (0, 256)
           if B * S * H < 1 << 20]


def test_window_asks_for_what_it_says(lib):
    asked = 0
    for B, S, T, H, Hk, d, w, n, chunk in WINDOWS:
        opt = ctypes.byref(_lib.SiOptions(chunk, 0, 0, 0, 0))
        need = window_size(lib, B, S, T, H, Hk, d, w, n, opt)
        if need == 0:
            continue
        asked += 1

        def call(ws, size):
            return lib.si_window_attention(FAKE, FAKE, FAKE, FAKE, None, B, S, T, H, Hk, d, w, n, 0.1, FAKE, None, opt, ws, size, None)

        assert call(FAKE, need - 1) == -5 and call(None, need) == -5 and call(ODD, need) == -4, (B, S, T, H, Hk, d, w, n, chunk)
    assert asked > 100


def test_cache4_asks_for_what_it_says(lib):
    asked = 0
    for B, S, T, H, Hk, d, w, n, chunk in WINDOWS:
        if S > 40:
            continue
        opt = ctypes.byref(_lib.SiOptions(chunk, 0, 0, 0, 0))
        for topk in (0, 7, 2048):
            if topk and w < 10 ** 9:
                continue
            win, sinks = (0, 0) if topk or w == 10 ** 9 else (w, n)
            width = -(-T // 16)
            need = cache4_size(lib, width, 16, topk, B, S, H, Hk, d, win, sinks, opt)
            if need == 0:
                continue
            asked += 1

            def call(ws, size):
                return lib.si_cache4_attention(FAKE, FAKE, 4, FAKE, width, 16, FAKE, None, FAKE if topk else None, topk, B, S, H, Hk, d, win, sinks,
                                               0.1, 1.0, 1.0, FAKE, None, opt, ws, size, None)

            assert call(FAKE, need - 1) == -5 and call(None, need) == -5 and call(ODD, need) == -4, (B, S, T, H, Hk, d, topk, chunk)
    assert asked > 50
