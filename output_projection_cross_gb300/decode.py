"""Python binding of beam-search decoding: same names as the C ABI, argument marshalling only.

As in lossk.py, every function takes torch tensors on the GPU, passes their
pointers and element counts to the C entry point on the current CUDA stream
and raises :class:`LosskError` for any status other than 580.  These calls do
not synchronise: ids and lengths are checked on the device, and what was found
wrong there is read with ``lossk_device_status(ws)``.  So a decoding loop keeps
a workspace (:func:`decode_workspace`) and its output tensors and passes them
in; both are created here when left out.  All of a call's tensors have to be on
the current device (``ValueError`` otherwise).
"""
from __future__ import annotations

import importlib.util
import os

import torch

from . import build as _build
from .lossk import LosskError, _check, _dtype_code, _len, _ptr, _stream, lib


class _NotBuilt:
    """Stands for the module where it is not built: importing the package, for the losses, does not need it."""

    def __getattr__(self, name):
        raise ImportError(f"the decoding calls' module is not built ({_build.CALLS}); run `python "
                          f"output_projection_cross_gb300/build.py` with a Python that has its headers")


def _load_calls():
    """The module through which the calls are made (ctypes takes 2 us for the arguments of one)."""
    path = _build.CALLS
    if not os.path.exists(path):
        return _NotBuilt()
    spec = importlib.util.spec_from_file_location("_lossk_calls", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.load(_build.LIB)
    return m


_calls = _load_calls()
_int32 = torch.int32
KIND_BEAM_SELECT, KIND_CACHE, KIND_PAGED_ATTN = 0, 1, 2

__all__ = ["KIND_BEAM_SELECT", "KIND_CACHE", "KIND_PAGED_ATTN", "decode_workspace", "beam_buffers",
           "lossk_decode_workspace_bytes", "lossk_beam_select", "lossk_beam_gather", "lossk_cache_fork",
           "lossk_cache_reserve", "lossk_cache_free", "lossk_cache_compact", "lossk_cache_copy", "lossk_cache_write",
           "lossk_paged_attn"]


def lossk_decode_workspace_bytes(kind: int, a: int, b: int, c: int = 0, d: int = 0) -> int:
    return lib.lossk_decode_workspace_bytes(kind, a, b, c, d)


def decode_workspace(kind: int, a: int, b: int, c: int = 0, d: int = 0, device=None) -> torch.Tensor:
    """A zeroed workspace for the sizes of ``kind``: (batch, beams, vocab, n_out), (n_seq, n_pages)
    or (n_seq, n_q_heads, n_kv_heads, head_dim)."""
    nb = lib.lossk_decode_workspace_bytes(kind, a, b, c, d)
    if nb < 0:
        raise ValueError(f"no workspace of kind {kind} for the sizes {(a, b, c, d)}")
    return torch.zeros(nb, dtype=torch.uint8, device=device or "cuda")


# These calls take microseconds, so the checks below are kept to attribute reads: a decoding step
# makes several calls per layer, and building a stream object alone takes 3 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(stream, *tensors):
    """The CUDA stream handle, the given stream's or the current one, of a call on these tensors (None
    left out).  Launches go to the current device, so tensors and stream have to be on it."""
    index = _calls.device(*tensors)
    if index < 0 or index != _current_device() or (stream is not None and stream.device_index != index):
        on = sorted({str(t.device) for t in tensors if t is not None})
        raise ValueError(f"the tensors (on {', '.join(on)}), workspace among them, and the stream must be on the "
                         f"current CUDA device")
    if stream is not None or _raw_stream is None:
        return _stream(stream)
    return _raw_stream(index)


# What a call makes for itself it makes on its stream: zeroed there before the call's kernels, and, once
# it is dropped, its memory handed on to that stream's work alone, which comes after them.
def _new(stream, shape, dtype, device, zeros=False):
    with torch.cuda.stream(stream):
        return (torch.zeros if zeros else torch.empty)(shape, dtype=dtype, device=device)


def _new_workspace(stream, device, kind, *sizes):
    with torch.cuda.stream(stream):
        return decode_workspace(kind, *sizes, device=device)


def _on_gpu(t, name, dtype=None, contiguous=True):
    # (that it is on the GPU is seen to for all tensors of a call together, in _stream_of)
    if t is None:
        return
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")


def _ints(names, *tensors):
    """(address, elements) of each int32 tensor, flat; None is no elements at address 0."""
    r = _calls.spans(_int32, *tensors)
    if r is None:
        for t, name in zip(tensors, names):
            _on_gpu(t, name, _int32)
        raise ValueError(f"{', '.join(names)} must be CUDA tensors")
    return r


def _span(t) -> int:
    """Elements from a strided tensor's first to its last."""
    n = t.numel()
    if n == 0 or t.is_contiguous():
        return n
    span = 1
    for size, stride in zip(t.shape, t.stride()):
        span += (size - 1) * stride
    return span


def _packed(shape, strides, first) -> bool:
    """Whether dimensions first.. lie in memory one after another."""
    want = 1
    for i in range(len(shape) - 1, first - 1, -1):
        if shape[i] != 1 and strides[i] != want:
            return False
        want *= shape[i]
    return True


# ---- beams --------------------------------------------------------------------------

def beam_buffers(batch: int, n_out: int, device="cuda") -> dict:
    """The output tensors of lossk_beam_select."""
    def new(dtype):
        return torch.empty((batch, n_out), dtype=dtype, device=device)
    return {"parent": new(torch.int32), "token": new(torch.int64), "score": new(torch.float32),
            "finished": new(torch.uint8), "length": new(torch.int32)}


def lossk_beam_select(logits, scores, n_out, temperature=1.0, allow=None, finished=None, end_token=-1,
                      lengths=None, length_alpha=0.0, out=None, lse_out=None, ws=None, stream=None) -> dict:
    """logits [batch * beams, vocab] (rows may be strided), scores float [batch, beams].

    allow: int32 words [ceil(vocab / 32)], or [1 or batch * beams, ceil(vocab / 32)].
    Returns ``out`` (see :func:`beam_buffers`)."""
    if logits.dim() != 2 or scores.dim() != 2 or logits.stride(1) != 1 and logits.shape[1] > 1:
        raise ValueError("logits must be [batch * beams, vocab] with contiguous rows, scores [batch, beams]")
    rows, V = logits.shape
    batch, beams = scores.shape
    if rows != batch * beams:
        raise ValueError(f"{rows} rows of logits for scores of shape {tuple(scores.shape)}")
    _on_gpu(logits, "logits", contiguous=False)
    _on_gpu(scores, "scores", torch.float32)
    _on_gpu(finished, "finished", torch.uint8)
    _on_gpu(lengths, "lengths", torch.int32)
    for t, nm in ((finished, "finished"), (lengths, "lengths")):
        if t is not None and t.numel() != rows:
            raise ValueError(f"{nm} must hold one value per beam")
    allow_stride = 0
    if allow is not None:
        _on_gpu(allow, "allow", torch.int32)
        if allow.dim() == 2 and allow.shape[0] > 1:
            if allow.shape[0] != rows:
                raise ValueError("allow must hold one mask, or one per row of logits")
            allow_stride = allow.shape[1]
    if out is None:
        with torch.cuda.stream(stream):
            out = beam_buffers(batch, n_out, logits.device)
    parent, token, score, done, length = out["parent"], out["token"], out["score"], out["finished"], out["length"]
    _on_gpu(parent, "parent", torch.int32)
    _on_gpu(token, "token", torch.int64)
    _on_gpu(score, "score", torch.float32)
    _on_gpu(done, "finished", torch.uint8)
    _on_gpu(length, "length", torch.int32)
    n = batch * n_out
    if not (parent.numel() == token.numel() == score.numel() == done.numel() == length.numel() == n):
        raise ValueError("out must hold tensors of [batch, n_out]")
    _on_gpu(lse_out, "lse_out", torch.float32)
    if lse_out is not None and lse_out.numel() != rows:
        raise ValueError("lse_out must hold one value per row of logits")
    if ws is None:
        ws = _new_workspace(stream, logits.device, KIND_BEAM_SELECT, batch, beams, V, n_out)
    stream = _stream_of(stream, logits, scores, allow, finished, lengths, parent, token, score, done, length,
                        lse_out, ws)
    st = _calls.lossk_beam_select(batch, beams, V, n_out, _dtype_code(logits), logits.data_ptr(), _span(logits),
                               logits.stride(0) if rows > 1 else max(V, 1), scores.data_ptr(), rows, temperature,
                               _ptr(allow), _len(allow), allow_stride, _ptr(finished), end_token, _ptr(lengths),
                               length_alpha, parent.data_ptr(), token.data_ptr(), score.data_ptr(), done.data_ptr(),
                               length.data_ptr(), _ptr(lse_out), ws.data_ptr(), ws.numel(), stream)
    _check(st, "lossk_beam_select")
    return out


def lossk_beam_gather(src, parent, dst=None, ws=None, stream=None):
    """dst[g, j] = src[g, parent[g, j]]; zeros where the parent is -1.  src [groups, n_src, ...]."""
    _on_gpu(src, "src")
    _on_gpu(parent, "parent", torch.int32)
    if parent.dim() != 2 or src.dim() < 2 or parent.shape[0] != src.shape[0]:
        raise ValueError("src must be [groups, n_src, ...], parent [groups, n_dst]")
    G, n_src = src.shape[:2]
    n_dst = parent.shape[1]
    if dst is None:
        dst = _new(stream, (G, n_dst) + tuple(src.shape[2:]), src.dtype, src.device)
    _on_gpu(dst, "dst", src.dtype)
    row = src.numel() * src.element_size() // max(G * n_src, 1)
    if ws is None:
        ws = _new(stream, 256, torch.uint8, src.device, zeros=True)
    stream = _stream_of(stream, parent, src, dst, ws)
    st = _calls.lossk_beam_gather(G, n_src, n_dst, row, parent.data_ptr(), parent.numel(), src.data_ptr(),
                               src.numel() * src.element_size(), dst.data_ptr(), dst.numel() * dst.element_size(),
                               ws.data_ptr(), ws.numel(), stream)
    _check(st, "lossk_beam_gather")
    return dst


# ---- the cache's pages ------------------------------------------------------------------

def _table(table, name="table"):
    """(rows, entries per row, row stride, elements) of a table, whose rows may be strided."""
    _on_gpu(table, name, torch.int32, contiguous=False)
    shape = table.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be [n_seq, max_pages]")
    n, m = shape
    if table.is_contiguous():
        return n, m, max(m, 1), n * m
    stride, one = table.stride()
    if m > 1 and one != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return n, m, stride if n > 1 else max(m, 1), _span(table)


def _pool(pool, pages):
    """(address, bytes, planes, plane stride, page stride, page bytes) of a pool [planes, pages, ...]."""
    _on_gpu(pool, "pool", contiguous=False)
    shape, strides, es = pool.shape, pool.stride(), pool.element_size()
    if len(shape) < 3 or not (pool.is_contiguous() or _packed(shape, strides, 2)):
        raise ValueError("pool must be [planes, pages, ...] with contiguous pages")
    if shape[1] != pages:
        raise ValueError(f"a pool of {shape[1]} pages with {pages} counts")
    page = pool.numel() * es // max(shape[0] * shape[1], 1)
    return (pool.data_ptr(), _span(pool) * es, shape[0], strides[0] * es if shape[0] > 1 else 0,
            strides[1] * es if pages > 1 else page, page)


def lossk_cache_fork(parent, table, lens, ref, page_size, table_out=None, lens_out=None, ws=None, stream=None):
    """parent int32 [groups, n_dst]; table holds groups * n_src rows.  Returns (table_out, lens_out)."""
    G, n_dst = parent.shape
    if lens_out is None:
        lens_out = _new(stream, G * n_dst, torch.int32, table.device)
    parents, parents_len, lengths, lengths_len, refs, pages, outs, outs_len = _ints(
        ("parent", "lens", "ref", "lens_out"), parent, lens, ref, lens_out)
    n, m, stride, table_len = _table(table)
    if n % G or lengths_len != n:
        raise ValueError(f"{n} rows and {lengths_len} lengths in {G} groups")
    if table_out is None:
        table_out = _new(stream, (G * n_dst, m), torch.int32, table.device)
    no, mo, stride_out, out_len = _table(table_out, "table_out")
    if no != G * n_dst or mo != m:
        raise ValueError("table_out must be [groups * n_dst, max_pages]")
    if ws is None:
        ws = _new_workspace(stream, table.device, KIND_CACHE, max(n, no), pages)
    stream = _stream_of(stream, parent, table, lens, ref, table_out, lens_out, ws)
    st = _calls.lossk_cache_fork(G, n // G, n_dst, m, page_size, pages, parents, parents_len, table.data_ptr(),
                                 table_len, stride, lengths, n, refs, pages, table_out.data_ptr(), out_len,
                                 stride_out, outs, outs_len, ws.data_ptr(), ws.numel(), stream)
    _check(st, "lossk_cache_fork")
    return table_out, lens_out


def lossk_cache_reserve(table, lens, ref, pool, page_size, n_new=1, ws=None, stream=None) -> None:
    """n_new: tokens to come for every sequence, or an int32 tensor with one count each."""
    each = n_new if isinstance(n_new, torch.Tensor) else None
    lengths, lengths_len, refs, pages, new, new_len = _ints(("lens", "ref", "n_new"), lens, ref, each)
    n, m, stride, table_len = _table(table)
    P = _pool(pool, pages)
    if ws is None:
        ws = _new_workspace(stream, table.device, KIND_CACHE, n, pages)
    stream = _stream_of(stream, each, table, lens, ref, pool, ws)
    st = _calls.lossk_cache_reserve(n, m, page_size, pages, 0 if each is not None else n_new, new, new_len,
                                    table.data_ptr(), table_len, stride, lengths, lengths_len, refs, pages, *P,
                                    ws.data_ptr(), ws.numel(), stream)
    _check(st, "lossk_cache_reserve")


def lossk_cache_free(table, lens, ref, page_size, drop=None, ws=None, stream=None) -> None:
    """drop: uint8 [n_seq], nonzero where the sequence goes (None: all)."""
    lengths, lengths_len, refs, pages = _ints(("lens", "ref"), lens, ref)
    _on_gpu(drop, "drop", torch.uint8)
    n, m, stride, table_len = _table(table)
    if ws is None:
        ws = _new_workspace(stream, table.device, KIND_CACHE, n, pages)
    stream = _stream_of(stream, drop, table, lens, ref, ws)
    st = _calls.lossk_cache_free(n, m, page_size, pages, _ptr(drop), _len(drop), table.data_ptr(), table_len, stride,
                                 lengths, lengths_len, refs, pages, ws.data_ptr(), ws.numel(),
                                 stream)
    _check(st, "lossk_cache_free")


def lossk_cache_compact(table, lens, ref, pool, page_size, table_out=None, ref_out=None, n_live_out=None, ws=None,
                        stream=None):
    """Returns (table_out, ref_out, n_live_out); the pool's live pages are in front then."""
    ref_out = ref_out if ref_out is not None else _new(stream, ref.shape, torch.int32, ref.device)
    n_live_out = n_live_out if n_live_out is not None else _new(stream, 1, torch.int32, ref.device)
    lengths, lengths_len, refs, pages, refs_out, refs_out_len, live, live_len = _ints(
        ("lens", "ref", "ref_out", "n_live_out"), lens, ref, ref_out, n_live_out)
    n, m, stride, table_len = _table(table)
    P = _pool(pool, pages)
    table_out = table_out if table_out is not None else _new(stream, (n, m), torch.int32, table.device)
    no, mo, stride_out, out_len = _table(table_out, "table_out")
    if no != n or mo != m or live_len < 1:
        raise ValueError("table_out must be shaped like table, n_live_out hold one value")
    if ws is None:
        ws = _new_workspace(stream, table.device, KIND_CACHE, n, pages)
    stream = _stream_of(stream, table, lens, ref, table_out, ref_out, n_live_out, pool, ws)
    st = _calls.lossk_cache_compact(n, m, page_size, pages, table.data_ptr(), table_len, stride, lengths,
                                    lengths_len, refs, pages, table_out.data_ptr(), out_len, stride_out, refs_out,
                                    refs_out_len, live, *P, ws.data_ptr(), ws.numel(), stream)
    _check(st, "lossk_cache_compact")
    return table_out, ref_out, n_live_out


def lossk_cache_copy(src, dst, pool, ws=None, stream=None) -> None:
    """Page src[i] of the pool to page dst[i], in every plane."""
    _on_gpu(src, "src", torch.int32)
    _on_gpu(dst, "dst", torch.int32)
    P = _pool(pool, pool.shape[1])
    if src.numel() != dst.numel():
        raise ValueError("src and dst must list as many pages")
    ws = ws if ws is not None else _new(stream, 256, torch.uint8, pool.device, zeros=True)
    stream = _stream_of(stream, src, dst, pool, ws)
    st = _calls.lossk_cache_copy(src.numel(), pool.shape[1], src.data_ptr(), src.numel(), dst.data_ptr(), dst.numel(),
                              *P, ws.data_ptr(), ws.numel(), stream)
    _check(st, "lossk_cache_copy")


def _pages(k, v):
    """(shape, strides, elements) of one layer's key and value pages [pages, page, heads, head_dim],
    whose elements of a head are contiguous."""
    _on_gpu(k, "k_pages", contiguous=False)
    _on_gpu(v, "v_pages", k.dtype, contiguous=False)
    shape, strides = k.shape, k.stride()
    if len(shape) != 4 or shape != v.shape or strides != v.stride() or (shape[3] > 1 and strides[3] != 1):
        raise ValueError("k_pages and v_pages must be [pages, page, heads, head_dim], laid out alike, heads contiguous")
    return shape, strides, _span(k)


def lossk_cache_write(k_new, v_new, k_pages, v_pages, table, lens, first=None, ws=None, stream=None) -> None:
    """k_new, v_new [n_tok, heads, head_dim] (tokens may be strided) into one layer's pages
    [pages, page, heads, head_dim] (any strides).  first: int32 [n_seq + 1], where each sequence's
    rows begin (None: one row per sequence)."""
    (n_pages, page, kv, hd), (sp, stok, sh, _), pages_len = _pages(k_pages, v_pages)
    lengths, lengths_len, firsts, firsts_len = _ints(("lens", "first"), lens, first)
    n, m, stride, table_len = _table(table)
    _on_gpu(k_new, "k_new", k_pages.dtype, contiguous=False)
    _on_gpu(v_new, "v_new", k_pages.dtype, contiguous=False)
    shape, strides = k_new.shape, k_new.stride()
    if len(shape) != 3 or shape[1] != kv or shape[2] != hd or not (k_new.is_contiguous() or _packed(shape, strides, 1)):
        raise ValueError("k_new must be [n_tok, heads, head_dim] with contiguous tokens")
    if shape != v_new.shape or strides != v_new.stride():
        raise ValueError("k_new and v_new must be laid out alike")
    n_tok = shape[0]
    ws = ws if ws is not None else _new(stream, 256, torch.uint8, table.device, zeros=True)
    stream = _stream_of(stream, k_new, v_new, k_pages, v_pages, table, lens, first, ws)
    st = _calls.lossk_cache_write(n_tok, n, kv, hd, m, page, n_pages, _dtype_code(k_pages), k_new.data_ptr(),
                               v_new.data_ptr(), _span(k_new), strides[0] if n_tok > 1 else kv * hd,
                               k_pages.data_ptr(), v_pages.data_ptr(), pages_len, sp, stok, sh,
                               table.data_ptr(), table_len, stride, lengths, lengths_len, firsts, firsts_len,
                               ws.data_ptr(), ws.numel(), stream)
    _check(st, "lossk_cache_write")


# ---- attention of one new token ------------------------------------------------------------

def lossk_paged_attn(q, k_pages, v_pages, table, lens, scale=None, window=0, share=1, max_len=0, out=None,
                     lse_out=None, ws=None, stream=None):
    """q [n_seq, n_q_heads, head_dim] (sequences may be strided) over one layer's pages
    [pages, page, heads, head_dim] (any strides).  scale defaults to head_dim ** -0.5; share: how
    many consecutive sequences may share leading pages.  Returns out."""
    (n_pages, page, kv, hd), (sp, stok, sh, _), pages_len = _pages(k_pages, v_pages)
    lengths, lengths_len = _ints(("lens",), lens)
    _on_gpu(q, "q", k_pages.dtype, contiguous=False)
    n, m, stride, table_len = _table(table)
    shape, strides = q.shape, q.stride()
    if len(shape) != 3 or shape[0] != n or shape[2] != hd or not (q.is_contiguous() or _packed(shape, strides, 1)):
        raise ValueError("q must be [n_seq, n_q_heads, head_dim] with contiguous sequences")
    hq = shape[1]
    if out is None:
        out = _new(stream, (n, hq, hd), q.dtype, q.device)
    _on_gpu(out, "out", q.dtype)
    _on_gpu(lse_out, "lse_out", torch.float32)
    if lse_out is not None and lse_out.numel() != n * hq:
        raise ValueError("lse_out must be [n_seq, n_q_heads]")
    if ws is None:
        ws = _new_workspace(stream, q.device, KIND_PAGED_ATTN, n, hq, kv, hd)
    stream = _stream_of(stream, q, k_pages, v_pages, table, lens, out, lse_out, ws)
    st = _calls.lossk_paged_attn(n, hq, kv, hd, m, page, n_pages, share, _dtype_code(q), q.data_ptr(), _span(q),
                              strides[0] if n > 1 else hq * hd, k_pages.data_ptr(), v_pages.data_ptr(), pages_len,
                              sp, stok, sh, table.data_ptr(), table_len, stride, lengths, lengths_len,
                              max_len, window, hd ** -0.5 if scale is None else scale, out.data_ptr(), out.numel(),
                              _ptr(lse_out), ws.data_ptr(), ws.numel(), stream)
    _check(st, "lossk_paged_attn")
    return out
