"""The cache calls of the C ABI refuse bad arguments on the host, before anything is launched (every
call here fails, or only asks for a size)."""

import ctypes

import pytest

from streaming_top_lightning_b200 import _lib, build

FAKE = ctypes.c_void_p(4096)   # aligned, never read: each call fails first
ODD = ctypes.c_void_p(4098)    # neither 16- nor 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def size():
    return ctypes.c_size_t(0)


def window(lib, B=1, S=1, T=100, H=8, Hk=2, d=128, w=64, n=4, scale=0.1, q=FAKE, k=FAKE, v=FAKE, lens=None, out=FAKE, lse=None,
           opt=None, ws=None, ws_bytes=0):
    return lib.si_window_attention(q, k, v, lens, None, B, S, T, H, Hk, d, w, n, scale, out, lse, opt, ws, ws_bytes, None)


def test_window_refusals(lib):
    for name in ("q", "k", "v", "out"):
        assert window(lib, **{name: None}) == -1, name
    for bad in (dict(B=0), dict(S=0), dict(T=0), dict(H=0), dict(Hk=0), dict(H=7), dict(d=96), dict(d=256), dict(T=1 << 30),
                dict(B=1 << 20, S=1 << 12), dict(B=1 << 20, T=1 << 12), dict(B=-1), dict(Hk=-2)):
        assert window(lib, **bad) == -2, bad
    for bad in (dict(w=0), dict(w=-5), dict(n=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-0.1)):
        assert window(lib, **bad) == -8, bad
    for name in ("q", "k", "v", "out", "lens", "lse"):
        assert window(lib, **{name: ODD}) == -4, name
    bad = _lib.SiOptions(100, 0, 0, 0, 0)
    assert window(lib, opt=ctypes.byref(bad)) == -8
    # many keys for one row: several CTAs, partial results
    n = size()
    assert lib.si_window_attention_workspace_size(1, 1, 100000, 8, 8, 128, 90000, 0, None, ctypes.byref(n)) == 0 and n.value > 0
    assert window(lib, T=100000, H=8, Hk=8, w=90000) == -5
    assert window(lib, T=100000, H=8, Hk=8, w=90000, ws=FAKE, ws_bytes=n.value - 1) == -5
    assert window(lib, T=100000, H=8, Hk=8, w=90000, ws=ctypes.c_void_p(4100), ws_bytes=n.value) == -4
    # a prompt needs none
    assert lib.si_window_attention_workspace_size(2, 4096, 4096, 64, 8, 128, 1024, 4, None, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.si_window_attention_workspace_size(1, 1, 1, 1, 1, 64, 1, 0, None, None) == -1


def test_page_bytes(lib):
    n = size()
    for heads, dim, page, want in ((1, 64, 16, 1152), (8, 128, 64, 73728), (3, 128, 256, 110592)):
        assert lib.si_cache4_page_bytes(heads, dim, page, ctypes.byref(n)) == 0 and n.value == want
    for bad in ((0, 64, 16), (1, 96, 16), (1, 64, 8), (1, 64, 48), (1, 64, 512), (1, 64, 0), (-1, 64, 16), (1, 64, -16)):
        assert lib.si_cache4_page_bytes(*bad, ctypes.byref(n)) == -2, bad
    assert lib.si_cache4_page_bytes(1, 64, 16, None) == -1


@pytest.mark.parametrize("call", ["si_cache4_append", "si_cache4_read"])
def test_row_refusals(lib, call):
    def run(k=FAKE, v=FAKE, B=1, S=1, Hk=1, d=64, pages=FAKE, n=4, table=FAKE, width=4, page=16, lens=FAKE, q_lens=None, ks=1.0, vs=1.0):
        return getattr(lib, call)(k, v, B, S, Hk, d, pages, n, table, width, page, lens, q_lens, ks, vs, None)

    for name in ("k", "v", "pages", "table", "lens"):
        assert run(**{name: None}) == -1, name
        assert run(**{name: ODD}) == -4, name
    assert run(q_lens=ODD) == -4
    for bad in (dict(B=0), dict(S=0), dict(Hk=0), dict(d=32), dict(n=0), dict(width=0), dict(page=24), dict(page=512), dict(width=1 << 26),
                dict(B=1 << 20, S=1 << 11)):
        assert run(**bad) == -2, bad
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 61, 2.0 ** -61):
        assert run(ks=bad) == -8 and run(vs=bad) == -8, bad


def test_cache4_attention_refusals(lib):
    def run(q=FAKE, pages=FAKE, n=4, table=FAKE, width=4, page=16, lens=FAKE, q_lens=None, idx=None, topk=0, B=1, S=1, H=8, Hk=2, d=64, w=0,
            sinks=0, scale=0.1, ks=1.0, vs=1.0, out=FAKE, lse=None, ws=None, ws_bytes=0):
        return lib.si_cache4_attention(q, pages, n, table, width, page, lens, q_lens, idx, topk, B, S, H, Hk, d, w, sinks, scale, ks, vs, out,
                                       lse, None, ws, ws_bytes, None)

    for name in ("q", "pages", "table", "lens", "out"):
        assert run(**{name: None}) == -1, name
        assert run(**{name: ODD}) == -4, name
    for name in ("q_lens", "lse"):
        assert run(**{name: ODD}) == -4, name
    assert run(idx=ODD, topk=4) == -4
    for bad in (dict(n=0), dict(page=20), dict(width=0), dict(H=9), dict(d=100), dict(B=0), dict(S=-1), dict(width=1 << 27)):
        assert run(**bad) == -2, bad
    for bad in (dict(idx=FAKE, topk=0), dict(idx=FAKE, topk=2049), dict(topk=5), dict(idx=FAKE, topk=-1)):
        assert run(**bad) == -3, bad
    for bad in (dict(w=-1), dict(sinks=3), dict(w=4, sinks=-1), dict(idx=FAKE, topk=4, w=8), dict(scale=-1.0), dict(ks=0.0), dict(vs=1e30)):
        assert run(**bad) == -8, bad
    n = size()
    assert lib.si_cache4_attention_workspace_size(1000, 128, 0, 1, 1, 8, 8, 128, 0, 0, None, ctypes.byref(n)) == 0 and n.value > 0
    assert run(width=1000, page=128, H=8, Hk=8, d=128) == -5


def test_page_call_refusals(lib):
    n = size()
    assert lib.si_cache_workspace_size(100, 4, 8, ctypes.byref(n)) == 0 and n.value > 0
    big = n.value
    for bad in ((0, 1, 0), (1, 0, 0), (1, 1, -1)):
        assert lib.si_cache_workspace_size(*bad, ctypes.byref(n)) == -2
    assert lib.si_cache_workspace_size(1, 1, 1, None) == -1

    def extend(refs=FAKE, n=100, table=FAKE, B=4, width=4, lens=FAKE, page=16, missing=FAKE, ws=FAKE, ws_bytes=big):
        return lib.si_cache_extend(refs, n, table, B, width, lens, page, missing, ws, ws_bytes, None)

    def fork(pages=FAKE, size=64, refs=FAKE, n=100, table=FAKE, B=4, width=4, lens=FAKE, src=FAKE, dst=FAKE, k=8, page=16, missing=FAKE, ws=FAKE,
             ws_bytes=big):
        return lib.si_cache_fork(pages, size, refs, n, table, B, width, lens, src, dst, k, page, missing, ws, ws_bytes, None)

    def free(refs=FAKE, n=100, table=FAKE, B=4, width=4, lens=FAKE, rows=FAKE, k=2):
        return lib.si_cache_free(refs, n, table, B, width, lens, rows, k, None)

    def compact(pages=FAKE, size=64, refs=FAKE, n=100, table=FAKE, B=4, width=4, ro=FAKE, to=FAKE, live=FAKE, ws=FAKE, ws_bytes=big):
        return lib.si_cache_compact(pages, size, refs, n, table, B, width, ro, to, live, ws, ws_bytes, None)

    for call, names in ((extend, "refs table lens missing"), (fork, "pages refs table lens src dst missing"), (free, "refs table lens rows"),
                        (compact, "pages refs table ro to live")):
        for name in names.split():
            assert call(**{name: None}) == -1, (call, name)
            assert call(**{name: ODD}) == -4, (call, name)
        for bad in (dict(n=0), dict(B=0), dict(width=0), dict(B=1 << 16, width=1 << 16)):
            assert call(**bad) == -2, (call, bad)
    for call in (extend, fork):
        for page in (0, 3, -4, 1 << 17):
            assert call(page=page) == -2
    for call in (fork, compact):
        for bytes_ in (0, 8, 24, -16, 1 << 31):
            assert call(size=bytes_) == -2
    for call in (extend, fork, compact):
        assert call(ws=None) == -5 and call(ws_bytes=64) == -5 and call(ws=ctypes.c_void_p(4104)) == -4
    assert fork(k=-1) == -2 and free(k=-1) == -2


def test_plan_is_the_same_for_the_size_and_the_call(lib):
    """Workspace sizes over many shapes: finite, and never shrinking as the keys grow."""
    n = size()
    for H, Hk in ((1, 1), (8, 2), (128, 1), (24, 8)):
        for B in (1, 7, 300):
            last = -1
            for width in (1, 3, 40, 500, 8000):
                assert lib.si_cache4_attention_workspace_size(width, 16, 0, B, 1, H, Hk, 128, 0, 0, None, ctypes.byref(n)) == 0
                assert 0 <= n.value < 4 << 30
                last = n.value
            assert last >= 0


def test_scales_that_overflow(lib):
    """A softmax scale has to be finite in log2 units and with the keys' scale in it."""
    assert window(lib, scale=3e38) == -8
    for scale, ks in ((3e38, 1.0), (1e25, 2.0 ** 60)):
        assert lib.si_cache4_attention(FAKE, FAKE, 4, FAKE, 4, 16, FAKE, None, None, 0, 1, 1, 8, 2, 64, 0, 0, scale, ks, 1.0, FAKE, None,
                                       None, None, 0, None) == -8
