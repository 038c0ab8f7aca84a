"""B200 (sm_100a) CSA lightning-indexer top-k.

Python face of libstreamindex.so.  It marshals torch CUDA tensors (device
pointers, the current stream) into the C ABI of include/streamindex.h; every
step of the computation runs in the library's CUDA kernels.  There is no CPU
path: the calls raise if the library is not built or no sm_100 GPU is present.

    idx, score = indexer_topk(q, w, kc, m=4, topk=512)

q [B,S,H_I,d_I] bf16, w [B,S,H_I] fp32, kc [B,S/m,d_I] bf16, all on one CUDA
device.  idx [B,S,topk] int32 (-1 padding), score [B,S,topk] fp32 (-inf padding).
"""

from __future__ import annotations

import ctypes
import functools

from . import _lib
from ._lib import SiOptions, SiPlanInfo, StreamIndexError  # noqa: F401

__all__ = [
    "indexer_topk", "indexer_topk_noalloc", "indexer_topk_fp8", "quantize_fp8_rows", "topk_scores",
    "workspace_size", "plan", "device_error", "options", "version", "StreamIndexError",
    "window_attention", "cache4_page_bytes", "cache4_append", "cache4_read", "cache4_attention",
    "cache_extend", "cache_fork", "cache_free", "cache_compact",
]


def _torch():
    import torch

    return torch


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None) -> ctypes.c_void_p:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, ndim, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


def options(key_chunk: int = 0, scratch_mb: int = 0, grid_ctas: int = 0, timeout_ms: int = 0,
            debug_flags: int = 0, score_events=None, row_finish: int = 0,
            key_tile: int = 0, strip_slots: int = 0, score_event_list=None,
            plan_heads: int = 0, plan_dim: int = 0, plan_fp8: int = 0) -> SiOptions:
    """Tuning knobs of include/streamindex.h.  ``score_events`` is an optional
    pair of ``torch.cuda.Event(enable_timing=True)`` that the call records around
    its score-kernel launches (on the call's stream); ``score_event_list`` a
    list of such events, recorded in pairs around each query block's score
    launch.  ``row_finish``: 1 = rows finished in the fused kernel, 2 = by the
    merge kernel, 0 = the library's choice.  ``key_tile``: keys per score strip
    (128 .. 1024; 0 = the library's choice); ``strip_slots``: score strips in
    flight (2..4; 0 = the library's choice).  ``plan_heads``/``plan_dim``/
    ``plan_fp8``: make ``topk_scores`` select with the fused kernel's plan for
    that indexer shape."""
    o = SiOptions(key_chunk, scratch_mb, grid_ctas, timeout_ms, debug_flags)
    o.row_finish = row_finish
    o.key_tile = key_tile
    o.strip_slots = strip_slots
    o.plan_heads = plan_heads
    o.plan_dim = plan_dim
    o.plan_fp8 = plan_fp8
    if score_events is not None:
        a, b = score_events
        o.score_events[0] = a.cuda_event
        o.score_events[1] = b.cuda_event
    if score_event_list:
        arr = (ctypes.c_void_p * len(score_event_list))(*[e.cuda_event for e in score_event_list])
        o._event_array = arr  # keep the array alive as long as the options
        o.score_event_list = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
        o.score_event_count = len(score_event_list)
    return o


def version() -> int:
    return _lib.load().si_version()


def workspace_size(B: int, S: int, H: int, D: int, m: int, topk: int, opts: SiOptions | None = None) -> int:
    n = ctypes.c_size_t(0)
    lib = _lib.load()
    _lib.check("si_indexer_topk_workspace_size",
               lib.si_indexer_topk_workspace_size(B, S, H, D, m, topk,
                                                  ctypes.byref(opts) if opts else None,
                                                  ctypes.byref(n)))
    return n.value


def plan(B: int, S: int, H: int, D: int, m: int, topk: int, fp8: bool = False,
         opts: SiOptions | None = None) -> dict:
    """The plan the library would run for this problem (si_indexer_topk_plan):
    tile shape, shared-memory plan, key chunks, query blocks and launches."""
    info = SiPlanInfo()
    lib = _lib.load()
    _lib.check("si_indexer_topk_plan",
               lib.si_indexer_topk_plan(B, S, H, D, m, topk, 1 if fp8 else 0,
                                        ctypes.byref(opts) if opts else None,
                                        ctypes.byref(info)))
    return info.as_dict()


def _outputs(B, S, topk, device, out):
    torch = _torch()
    if out is not None:
        idx, score = out
        _need(idx, torch.int32, 3, "out_idx")
        _need(score, torch.float32, 3, "out_score")
        if tuple(idx.shape) != (B, S, topk) or tuple(score.shape) != (B, S, topk):
            raise ValueError("out tensors must be [B,S,topk]")
        return idx, score
    return (torch.empty((B, S, topk), dtype=torch.int32, device=device),
            torch.empty((B, S, topk), dtype=torch.float32, device=device))


def indexer_topk(q, w, kc, m: int, topk: int, *, out=None, opts: SiOptions | None = None,
                 workspace=None, stream=None):
    """Top-k compressed keys per query (bf16 score path).  Returns (idx, score)."""
    torch = _torch()
    _need(q, torch.bfloat16, 4, "q")
    _need(w, torch.float32, 3, "w")
    _need(kc, torch.bfloat16, 3, "kc")
    B, S, H, D = q.shape
    idx, score = _outputs(B, S, topk, q.device, out)
    lib = _lib.load()
    st = _stream(stream)
    if opts is None and workspace is None:
        rc = lib.si_indexer_topk(_ptr(q), _ptr(w), _ptr(kc), B, S, H, D, m, topk, _ptr(idx),
                                 _ptr(score), st)
        _lib.check("si_indexer_topk", rc)
        return idx, score
    need = workspace_size(B, S, H, D, m, topk, opts)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    rc = lib.si_indexer_topk_ex(_ptr(q), _ptr(w), _ptr(kc), B, S, H, D, m, topk, _ptr(idx),
                                _ptr(score), ctypes.byref(opts) if opts else None,
                                _ptr(workspace), workspace.numel(), st)
    _lib.check("si_indexer_topk_ex", rc)
    return idx, score


def decode_workspace_size(B: int, S_q: int, t0: int, T: int, H: int, D: int, m: int, topk: int,
                          opts: SiOptions | None = None) -> int:
    n = ctypes.c_size_t(0)
    lib = _lib.load()
    _lib.check("si_indexer_decode_workspace_size",
               lib.si_indexer_decode_workspace_size(B, S_q, t0, T, H, D, m, topk,
                                                    ctypes.byref(opts) if opts else None,
                                                    ctypes.byref(n)))
    return n.value


def decode_plan(B: int, S_q: int, t0: int, T: int, H: int, D: int, m: int, topk: int,
                opts: SiOptions | None = None) -> dict:
    """The plan si_indexer_decode would run (tile shape, key chunks, launches)."""
    info = SiPlanInfo()
    lib = _lib.load()
    _lib.check("si_indexer_decode_plan",
               lib.si_indexer_decode_plan(B, S_q, t0, T, H, D, m, topk,
                                          ctypes.byref(opts) if opts else None,
                                          ctypes.byref(info)))
    return info.as_dict()


def indexer_decode(q, w, kc, t0: int, m: int, topk: int, *, out=None,
                   opts: SiOptions | None = None, workspace=None, stream=None):
    """Top-k compressed keys for the queries at sequence positions t0 ..
    t0 + S_q - 1 (q [B,S_q,H,D] bf16, w [B,S_q,H] fp32) against the keys kc
    [B,T,D] bf16 compressed so far (si_indexer_decode).  Returns (idx, score),
    each [B,S_q,topk]."""
    torch = _torch()
    _need(q, torch.bfloat16, 4, "q")
    _need(w, torch.float32, 3, "w")
    _need(kc, torch.bfloat16, 3, "kc")
    B, S, H, D = q.shape
    T = kc.shape[1]
    idx, score = _outputs(B, S, topk, q.device, out)
    need = decode_workspace_size(B, S, t0, T, H, D, m, topk, opts)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    rc = _lib.load().si_indexer_decode(_ptr(q), _ptr(w), _ptr(kc), B, S, t0, T, H, D, m, topk,
                                       _ptr(idx), _ptr(score),
                                       ctypes.byref(opts) if opts else None, _ptr(workspace),
                                       workspace.numel(), _stream(stream))
    _lib.check("si_indexer_decode", rc)
    return idx, score


def pivot_workspace_size(B: int, S: int, H: int, D: int, m: int, topk: int, G: int, C: int,
                         opts: SiOptions | None = None) -> int:
    n = ctypes.c_size_t(0)
    lib = _lib.load()
    _lib.check("si_indexer_pivot_workspace_size",
               lib.si_indexer_pivot_workspace_size(B, S, H, D, m, topk, G, C,
                                                   ctypes.byref(opts) if opts else None,
                                                   ctypes.byref(n)))
    return n.value


def indexer_pivot(q, w, kc, m: int, topk: int, G: int, C: int, *, out=None,
                  opts: SiOptions | None = None, workspace=None, stream=None):
    """Query-group candidate scan (si_indexer_pivot): groups of G queries share
    their last query's C best keys as candidates.  Returns (idx, score)."""
    torch = _torch()
    _need(q, torch.bfloat16, 4, "q")
    _need(w, torch.float32, 3, "w")
    _need(kc, torch.bfloat16, 3, "kc")
    B, S, H, D = q.shape
    idx, score = _outputs(B, S, topk, q.device, out)
    need = pivot_workspace_size(B, S, H, D, m, topk, G, C, opts)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    rc = _lib.load().si_indexer_pivot(_ptr(q), _ptr(w), _ptr(kc), B, S, H, D, m, topk, G, C,
                                      _ptr(idx), _ptr(score), ctypes.byref(opts) if opts else None,
                                      _ptr(workspace), workspace.numel(), _stream(stream))
    _lib.check("si_indexer_pivot", rc)
    return idx, score


def sparse_attention(qa, ka, va, idx, scale: float | None = None, *, out=None,
                     opts: SiOptions | None = None, stream=None):
    """Multi-query attention of each query's heads over the entries its row of
    ``idx`` lists (si_sparse_attention): qa [B,S,128,128] bf16, ka and va
    [B,T,128] bf16, idx [B,S,topk] int32 (-1 padding).  ``scale`` defaults to
    1/sqrt(128).  Returns out [B,S,128,128] fp32."""
    torch = _torch()
    _need(qa, torch.bfloat16, 4, "qa")
    _need(ka, torch.bfloat16, 3, "ka")
    _need(va, torch.bfloat16, 3, "va")
    _need(idx, torch.int32, 3, "idx")
    B, S, H, D = qa.shape
    T = ka.shape[1]
    if tuple(va.shape) != tuple(ka.shape) or idx.shape[0] != B or idx.shape[1] != S:
        raise ValueError("ka, va must be [B,T,D] and idx [B,S,topk]")
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    if out is None:
        out = torch.empty((B, S, H, D), dtype=torch.float32, device=qa.device)
    _need(out, torch.float32, 4, "out")
    rc = _lib.load().si_sparse_attention(_ptr(qa), _ptr(ka), _ptr(va), _ptr(idx), B, S, T, H, D,
                                         idx.shape[2], float(scale), _ptr(out),
                                         ctypes.byref(opts) if opts else None, _stream(stream))
    _lib.check("si_sparse_attention", rc)
    return out


def indexer_topk_noalloc(q, w, kc, m: int, topk: int, *, out=None, stream=None):
    """``indexer_topk`` through the entry point that allocates no device memory
    (its scratch is a fixed array inside the library; see
    si_indexer_topk_noalloc in include/streamindex.h).  Returns (idx, score);
    pass ``out`` to avoid allocating the outputs here as well."""
    torch = _torch()
    _need(q, torch.bfloat16, 4, "q")
    _need(w, torch.float32, 3, "w")
    _need(kc, torch.bfloat16, 3, "kc")
    B, S, H, D = q.shape
    idx, score = _outputs(B, S, topk, q.device, out)
    rc = _lib.load().si_indexer_topk_noalloc(_ptr(q), _ptr(w), _ptr(kc), B, S, H, D, m, topk,
                                             _ptr(idx), _ptr(score), _stream(stream))
    _lib.check("si_indexer_topk_noalloc", rc)
    return idx, score


def indexer_topk_fp8(q8, s_q, w, k8, s_k, m: int, topk: int, *, out=None,
                     opts: SiOptions | None = None, workspace=None, stream=None):
    """FP8 (E4M3) score path: q8 [B,S,H,D] and k8 [B,T,D] uint8 codes with
    per-row scales s_q [B,S,H], s_k [B,T].  Returns (idx, score)."""
    torch = _torch()
    _need(q8, torch.uint8, 4, "q8")
    _need(s_q, torch.float32, 3, "s_q")
    _need(w, torch.float32, 3, "w")
    _need(k8, torch.uint8, 3, "k8")
    _need(s_k, torch.float32, 2, "s_k")
    B, S, H, D = q8.shape
    idx, score = _outputs(B, S, topk, q8.device, out)
    need = workspace_size(B, S, H, D, m, topk, opts)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q8.device)
    lib = _lib.load()
    rc = lib.si_indexer_topk_fp8(_ptr(q8), _ptr(s_q), _ptr(w), _ptr(k8), _ptr(s_k), B, S, H, D, m,
                                 topk, _ptr(idx), _ptr(score),
                                 ctypes.byref(opts) if opts else None, _ptr(workspace),
                                 workspace.numel(), _stream(stream))
    _lib.check("si_indexer_topk_fp8", rc)
    return idx, score


def quantize_fp8_rows(x, stream=None):
    """Per-row E4M3 quantisation of a bf16 tensor [..., cols]: returns
    (codes uint8 [..., cols], scale fp32 [...])."""
    torch = _torch()
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 CUDA tensor")
    cols = x.shape[-1]
    rows = x.numel() // cols
    x8 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rc = _lib.load().si_quantize_fp8_rows(_ptr(x), rows, cols, _ptr(x8), _ptr(scale),
                                          _stream(stream))
    _lib.check("si_quantize_fp8_rows", rc)
    return x8, scale


def topk_scores(scores, m: int, topk: int, *, out=None, opts: SiOptions | None = None,
                stream=None):
    """Selection alone on given fp32 scores [B,S,T] (causal rule with ratio m)."""
    torch = _torch()
    _need(scores, torch.float32, 3, "scores")
    B, S, T = scores.shape
    idx, score = _outputs(B, S, topk, scores.device, out)
    rc = _lib.load().si_topk_scores(_ptr(scores), B, S, T, m, topk, _ptr(idx), _ptr(score),
                                    ctypes.byref(opts) if opts else None, _stream(stream))
    _lib.check("si_topk_scores", rc)
    return idx, score


def device_error(stream=None) -> int:
    """Synchronise and return the device status word as an SI status code."""
    return _lib.load().si_get_last_device_error(_stream(stream))


# ---- key/value cache: window attention, 4-bit pages, the pages' life
#
# A decode step makes several of these calls per layer, so their checks are
# kept short: one comparison per tensor, plain integers to ctypes, and the
# device and stream contexts only where the call needs them.


def _elsewhere(t, stream) -> bool:
    """Whether a call on t has to change the current device or stream first."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("the call's tensors must be CUDA tensors")
    return stream is not None or t.get_device() != torch.cuda.current_device()


class _at:
    """The device of a call's tensors, whichever is current, and the stream it
    was given, whose memory the call's own tensors then come from."""

    def __init__(self, t, stream):
        torch = _torch()
        if stream is not None and stream.device != t.device:
            raise ValueError("the stream is on another device than the tensors")
        self.guards = [torch.cuda.device(t.device)]
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _raw_stream(index: int) -> int:
    return _torch()._C._cuda_getCurrentRawStream(index)


def _check(index, t, dtype, shape, name):
    """t is a contiguous tensor of this type and shape on device ``index``."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a CUDA tensor")
    if (t.get_device() != index or t.dtype != dtype or t.shape != shape
            or not t.is_contiguous()):
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, the call's tensors are on cuda:{index}")
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)}, got {t.dtype} "
                         f"{list(t.shape)} with strides {list(t.stride())}")


def _dims(t, n, name):
    if not isinstance(t, _torch().Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a {n}-d tensor")
    return t.shape


@functools.lru_cache(maxsize=4096)
def _sizes(name: str, *args) -> int:
    """A size that the library answers from whole numbers alone."""
    n = ctypes.c_size_t(0)
    _lib.check(name, getattr(_lib.load(), name)(*args, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=4096)
def _plan_size(index: int, name: str, *args) -> int:
    """A workspace size of device ``index``, the current one."""
    return _sizes.__wrapped__(name, *args)


def _planned(index, name, args, opts):
    """Workspace bytes of a call with options, which the caller may change from
    one call to the next; without them they depend on the sizes and the device."""
    if opts is None:
        return _plan_size(index, name, *args, None)
    n = ctypes.c_size_t(0)
    _lib.check(name, getattr(_lib.load(), name)(*args, ctypes.byref(opts), ctypes.byref(n)))
    return n.value


def _scratch(need, workspace, t):
    """The call's workspace as (tensor or None, address, bytes): the caller's,
    or one of its own."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        torch = _torch()
        workspace = torch.empty(need, dtype=torch.uint8, device=t.device)
    elif workspace.dtype != _torch().uint8 or workspace.get_device() != t.get_device() \
            or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the call's device")
    return workspace, workspace.data_ptr(), workspace.numel()


def _attention_out(index, qa, out, lse):
    torch = _torch()
    B, S, H, D = qa.shape
    if out is None:
        out = torch.empty((B, S, H, D), dtype=torch.bfloat16, device=qa.device)
    else:
        _check(index, out, torch.bfloat16, (B, S, H, D), "out")
    if lse is None:
        lse = torch.empty((B, S, H), dtype=torch.float32, device=qa.device)
    else:
        _check(index, lse, torch.float32, (B, S, H), "lse")
    return out, lse


def _address(index, t, B, name):
    """Address of an optional int32 [B] tensor."""
    if t is None:
        return None
    _check(index, t, _torch().int32, (B,), name)
    return t.data_ptr()


def window_attention(qa, ka, va, window: int, sinks: int = 0, *, lens=None, q_lens=None,
                     scale: float | None = None, out=None, lse=None,
                     opts: SiOptions | None = None, workspace=None, stream=None):
    """Attention of each query to the last ``window`` tokens up to its own and
    to the first ``sinks`` ones (si_window_attention): qa [B,S,H,D] bf16, ka and
    va [B,T,H_k,D] bf16, D 64 or 128, H a multiple of H_k.  ``lens`` [B] int32:
    tokens of each sequence (default T); ``q_lens`` [B] int32: how many of the
    S query rows it has (default S); they are its newest tokens.  ``scale``
    defaults to 1/sqrt(D).  Returns (out [B,S,H,D] bf16, lse [B,S,H] fp32: the
    logarithm of each row's sum of exponentials, which joins this result with
    another over other keys); rows past q_lens are left as they were."""
    if _elsewhere(qa, stream):
        with _at(qa, stream):
            return window_attention(qa, ka, va, window, sinks, lens=lens, q_lens=q_lens,
                                    scale=scale, out=out, lse=lse, opts=opts, workspace=workspace)
    bf16 = _torch().bfloat16
    at = qa.get_device()
    B, S, H, D = _dims(qa, 4, "qa")
    _, T, Hk, _ = _dims(ka, 4, "ka")
    _check(at, qa, bf16, (B, S, H, D), "qa")
    _check(at, ka, bf16, (B, T, Hk, D), "ka")
    _check(at, va, bf16, (B, T, Hk, D), "va")
    # the arguments stay referenced: a temporary's memory must not become the workspace's
    lens_at, q_lens_at = _address(at, lens, B, "lens"), _address(at, q_lens, B, "q_lens")
    need = _planned(at, "si_window_attention_workspace_size", (B, S, T, H, Hk, D, window, sinks), opts)
    out, lse = _attention_out(at, qa, out, lse)
    _keep, ws, ws_bytes = _scratch(need, workspace, qa)
    rc = _lib.load().si_window_attention(
        qa.data_ptr(), ka.data_ptr(), va.data_ptr(), lens_at, q_lens_at, B, S, T, H, Hk, D, window,
        sinks, D ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(),
        None if opts is None else ctypes.byref(opts), ws, ws_bytes, _raw_stream(at))
    if rc:
        _lib.check("si_window_attention", rc)
    return out, lse


def cache4_page_bytes(heads: int, dim: int, page: int) -> int:
    """Bytes of one page of a 4-bit cache (si_cache4_page_bytes): ``page`` tokens
    of ``heads`` kv heads of ``dim`` elements."""
    return _sizes("si_cache4_page_bytes", heads, dim, page)


def _cache4(at, pages, table, lens, B, heads, dim, page):
    """Checks a cache; its number of pages and its table's width."""
    torch = _torch()
    n = _dims(pages, 2, "pages")[0]
    width = _dims(table, 2, "table")[1]
    _check(at, pages, torch.uint8, (n, cache4_page_bytes(heads, dim, page)), "pages")
    _check(at, table, torch.int32, (B, width), "table")
    _check(at, lens, torch.int32, (B,), "lens")
    return n, width


def cache4_append(k, v, pages, table, lens, page: int, *, q_lens=None, k_scale: float = 1.0,
                  v_scale: float = 1.0, stream=None):
    """Round the newest tokens' key and value rows (k, v [B,S,H_k,D] bf16) into
    the 4-bit pages (si_cache4_append): row i < q_lens[b] is token
    lens[b] - q_lens[b] + i.  ``pages`` [n_pages, cache4_page_bytes] uint8,
    ``table`` [B,width] int32, ``lens`` [B] int32 with the new tokens counted."""
    if _elsewhere(k, stream):
        with _at(k, stream):
            return cache4_append(k, v, pages, table, lens, page, q_lens=q_lens, k_scale=k_scale,
                                 v_scale=v_scale)
    bf16 = _torch().bfloat16
    at = k.get_device()
    B, S, Hk, D = _dims(k, 4, "k")
    n, width = _cache4(at, pages, table, lens, B, Hk, D, page)
    _check(at, k, bf16, (B, S, Hk, D), "k")
    _check(at, v, bf16, (B, S, Hk, D), "v")
    rc = _lib.load().si_cache4_append(k.data_ptr(), v.data_ptr(), B, S, Hk, D, pages.data_ptr(), n,
                                      table.data_ptr(), width, page, lens.data_ptr(),
                                      _address(at, q_lens, B, "q_lens"), k_scale, v_scale,
                                      _raw_stream(at))
    if rc:
        _lib.check("si_cache4_append", rc)
    return pages


def cache4_read(pages, table, lens, S: int, heads: int, dim: int, page: int, *, q_lens=None,
                k_scale: float = 1.0, v_scale: float = 1.0, out=None, stream=None):
    """The newest tokens' rows back as bf16 (si_cache4_read): (k, v), each
    [B,S,heads,dim]; rows of tokens that are not in the cache are left as they
    were in ``out``."""
    if _elsewhere(pages, stream):
        with _at(pages, stream):
            return cache4_read(pages, table, lens, S, heads, dim, page, q_lens=q_lens,
                               k_scale=k_scale, v_scale=v_scale, out=out)
    torch = _torch()
    at = pages.get_device()
    B = _dims(table, 2, "table")[0]
    n, width = _cache4(at, pages, table, lens, B, heads, dim, page)
    if out is None:
        out = tuple(torch.empty((B, S, heads, dim), dtype=torch.bfloat16, device=pages.device)
                    for _ in range(2))
    k, v = out
    _check(at, k, torch.bfloat16, (B, S, heads, dim), "out[0]")
    _check(at, v, torch.bfloat16, (B, S, heads, dim), "out[1]")
    rc = _lib.load().si_cache4_read(k.data_ptr(), v.data_ptr(), B, S, heads, dim, pages.data_ptr(),
                                    n, table.data_ptr(), width, page, lens.data_ptr(),
                                    _address(at, q_lens, B, "q_lens"), k_scale, v_scale,
                                    _raw_stream(at))
    if rc:
        _lib.check("si_cache4_read", rc)
    return k, v


def cache4_attention(qa, pages, table, lens, heads: int, page: int, window: int = 0,
                     sinks: int = 0, *, q_lens=None, idx=None, scale: float | None = None,
                     k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None,
                     opts: SiOptions | None = None, workspace=None, stream=None):
    """Attention of the newest tokens' queries (qa [B,S,H,D] bf16) over a 4-bit
    cache of ``heads`` kv heads (si_cache4_attention): over every key up to the
    query's own (window 0), over a window and sinks as ``window_attention``, or
    over the entries that ``idx`` [B,S,topk] int32 lists (the rows of
    ``indexer_topk`` and ``indexer_decode``).  Returns (out, lse) as
    ``window_attention``."""
    if _elsewhere(qa, stream):
        with _at(qa, stream):
            return cache4_attention(qa, pages, table, lens, heads, page, window, sinks,
                                    q_lens=q_lens, idx=idx, scale=scale, k_scale=k_scale,
                                    v_scale=v_scale, out=out, lse=lse, opts=opts,
                                    workspace=workspace)
    torch = _torch()
    at = qa.get_device()
    B, S, H, D = _dims(qa, 4, "qa")
    n, width = _cache4(at, pages, table, lens, B, heads, D, page)
    _check(at, qa, torch.bfloat16, (B, S, H, D), "qa")
    topk, entries = 0, None
    if idx is not None:
        topk = _dims(idx, 3, "idx")[2]
        _check(at, idx, torch.int32, (B, S, topk), "idx")
        entries = idx.data_ptr()
    need = _planned(at, "si_cache4_attention_workspace_size",
                    (width, page, topk, B, S, H, heads, D, window, sinks), opts)
    out, lse = _attention_out(at, qa, out, lse)
    _keep, ws, ws_bytes = _scratch(need, workspace, qa)
    rc = _lib.load().si_cache4_attention(
        qa.data_ptr(), pages.data_ptr(), n, table.data_ptr(), width, page, lens.data_ptr(),
        _address(at, q_lens, B, "q_lens"), entries, topk, B, S, H, heads, D, window, sinks,
        D ** -0.5 if scale is None else scale, k_scale, v_scale, out.data_ptr(), lse.data_ptr(),
        None if opts is None else ctypes.byref(opts), ws, ws_bytes, _raw_stream(at))
    if rc:
        _lib.check("si_cache4_attention", rc)
    return out, lse


def _pool(refs, table, lens):
    """Checks a pool's state; its device, pages, rows and width."""
    int32 = _torch().int32
    at = refs.get_device()
    n, = _dims(refs, 1, "refs")
    B, width = _dims(table, 2, "table")
    _check(at, refs, int32, (n,), "refs")
    _check(at, table, int32, (B, width), "table")
    if lens is not None:
        _check(at, lens, int32, (B,), "lens")
    return at, n, B, width


def cache_extend(refs, table, lens, page: int, *, workspace=None, stream=None):
    """Give each row of ``table`` [B,width] the pages that it lacks for lens[b]
    tokens, the lowest free ones first (si_cache_extend); ``refs`` [n_pages]
    counts each page's holders.  Returns an int32 [1] tensor: entries for which
    no page was free."""
    if _elsewhere(refs, stream):
        with _at(refs, stream):
            return cache_extend(refs, table, lens, page, workspace=workspace)
    at, n, B, width = _pool(refs, table, lens)
    missing = refs.new_empty(1)
    _keep, ws, ws_bytes = _scratch(_sizes("si_cache_workspace_size", n, B, 0), workspace, refs)
    rc = _lib.load().si_cache_extend(refs.data_ptr(), n, table.data_ptr(), B, width,
                                     lens.data_ptr(), page, missing.data_ptr(), ws, ws_bytes,
                                     _raw_stream(at))
    if rc:
        _lib.check("si_cache_extend", rc)
    return missing


def cache_fork(pages, refs, table, lens, src, dst, page: int, *, workspace=None, stream=None):
    """Make each row dst[i] a copy of row src[i] (si_cache_fork): whole pages are
    shared, a partly filled last one is copied.  The rows dst must be empty
    (``cache_free``).  Returns an int32 [1] tensor: children not made."""
    if _elsewhere(refs, stream):
        with _at(refs, stream):
            return cache_fork(pages, refs, table, lens, src, dst, page, workspace=workspace)
    torch = _torch()
    at, n, B, width = _pool(refs, table, lens)
    size = _dims(pages, 2, "pages")[1]
    _check(at, pages, torch.uint8, (n, size), "pages")
    count, = _dims(src, 1, "src")
    _check(at, src, torch.int32, (count,), "src")
    _check(at, dst, torch.int32, (count,), "dst")
    missing = refs.new_empty(1)
    _keep, ws, ws_bytes = _scratch(_sizes("si_cache_workspace_size", n, B, count), workspace, refs)
    rc = _lib.load().si_cache_fork(pages.data_ptr(), size, refs.data_ptr(), n, table.data_ptr(), B,
                                   width, lens.data_ptr(), src.data_ptr(), dst.data_ptr(), count,
                                   page, missing.data_ptr(), ws, ws_bytes, _raw_stream(at))
    if rc:
        _lib.check("si_cache_fork", rc)
    return missing


def cache_free(refs, table, lens, rows, *, stream=None):
    """Empty the listed rows: their pages lose a holder (si_cache_free)."""
    if _elsewhere(refs, stream):
        with _at(refs, stream):
            return cache_free(refs, table, lens, rows)
    at, n, B, width = _pool(refs, table, lens)
    count, = _dims(rows, 1, "rows")
    _check(at, rows, _torch().int32, (count,), "rows")
    rc = _lib.load().si_cache_free(refs.data_ptr(), n, table.data_ptr(), B, width, lens.data_ptr(),
                                   rows.data_ptr(), count, _raw_stream(at))
    if rc:
        _lib.check("si_cache_free", rc)


def cache_compact(pages, refs, table, *, out=None, workspace=None, stream=None):
    """Move the pages in use to the front of the pool (si_cache_compact).
    Returns (table, refs, live): the new table and counts (``out`` = (table,
    refs) to write them in place, else new tensors) and an int32 [1] tensor with
    the number of pages in use."""
    if _elsewhere(refs, stream):
        with _at(refs, stream):
            return cache_compact(pages, refs, table, out=out, workspace=workspace)
    torch = _torch()
    at, n, B, width = _pool(refs, table, None)
    size = _dims(pages, 2, "pages")[1]
    _check(at, pages, torch.uint8, (n, size), "pages")
    if out is None:
        out = (torch.empty_like(table), torch.empty_like(refs))
    new_table, new_refs = out
    _check(at, new_table, torch.int32, (B, width), "out[0]")
    _check(at, new_refs, torch.int32, (n,), "out[1]")
    live = refs.new_empty(1)
    _keep, ws, ws_bytes = _scratch(_sizes("si_cache_workspace_size", n, B, 0), workspace, refs)
    rc = _lib.load().si_cache_compact(pages.data_ptr(), size, refs.data_ptr(), n, table.data_ptr(),
                                      B, width, new_refs.data_ptr(), new_table.data_ptr(),
                                      live.data_ptr(), ws, ws_bytes, _raw_stream(at))
    if rc:
        _lib.check("si_cache_compact", rc)
    return new_table, new_refs, live
