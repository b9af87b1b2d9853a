"""Python binding of beam-search decoding: same names as the C ABI, argument marshalling only.

As in lossk.py, every function takes torch tensors on the GPU, passes their
pointers and element counts to the C entry point on the current CUDA stream
and raises :class:`LosskError` for any status other than 580.  These calls do
not synchronise: ids and lengths are checked on the device, and what was found
wrong there is read with ``lossk_device_status(ws)``.  So a decoding loop keeps
a workspace (:func:`decode_workspace`) and its output tensors and passes them
in; both are created here when left out.
"""
from __future__ import annotations

import torch

from .lossk import LosskError, _check, _dtype_code, _len, _ptr, _stream, lib

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


def _on_gpu(t, name, dtype=None, contiguous=True):
    if t is None:
        return
    if not t.is_cuda or (contiguous and not t.is_contiguous()):
        raise ValueError(f"{name} must be a {'contiguous ' if contiguous else ''}CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")


def _span(t) -> int:
    """Elements from a strided tensor's first to its last."""
    return 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())) if t.numel() else 0


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
        out = beam_buffers(batch, n_out, logits.device)
    for key, dtype in (("parent", torch.int32), ("token", torch.int64), ("score", torch.float32),
                       ("finished", torch.uint8), ("length", torch.int32)):
        t = out[key]
        _on_gpu(t, key, dtype)
        if t.numel() != batch * n_out:
            raise ValueError(f"out[{key!r}] must be [batch, n_out]")
    _on_gpu(lse_out, "lse_out", torch.float32)
    if lse_out is not None and lse_out.numel() != rows:
        raise ValueError("lse_out must hold one value per row of logits")
    if ws is None:
        ws = decode_workspace(KIND_BEAM_SELECT, batch, beams, V, n_out, logits.device)
    st = lib.lossk_beam_select(batch, beams, V, n_out, _dtype_code(logits), logits.data_ptr(), _span(logits),
                               logits.stride(0) if rows > 1 else max(V, 1), scores.data_ptr(), rows, temperature,
                               _ptr(allow), _len(allow), allow_stride, _ptr(finished), end_token, _ptr(lengths),
                               length_alpha, out["parent"].data_ptr(), out["token"].data_ptr(),
                               out["score"].data_ptr(), out["finished"].data_ptr(), out["length"].data_ptr(),
                               _ptr(lse_out), ws.data_ptr(), ws.numel(), _stream(stream))
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
        dst = torch.empty((G, n_dst) + tuple(src.shape[2:]), dtype=src.dtype, device=src.device)
    _on_gpu(dst, "dst", src.dtype)
    row = src[0, 0].numel() * src.element_size() if src.numel() else 0
    if ws is None:
        ws = torch.zeros(256, dtype=torch.uint8, device=src.device)
    st = lib.lossk_beam_gather(G, n_src, n_dst, row, parent.data_ptr(), parent.numel(), src.data_ptr(),
                               src.numel() * src.element_size(), dst.data_ptr(), dst.numel() * dst.element_size(),
                               ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "lossk_beam_gather")
    return dst


# ---- the cache's pages ------------------------------------------------------------------

def _ints(**named):
    for nm, t in named.items():
        _on_gpu(t, nm, torch.int32)


def _table(table, name="table"):
    """(rows, entries per row, row stride) of a table, whose rows may be strided."""
    _on_gpu(table, name, torch.int32, contiguous=False)
    if table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"{name} must be [n_seq, max_pages] with contiguous rows")
    n, m = table.shape
    return n, m, table.stride(0) if n > 1 else max(m, 1)


def _pool(pool):
    """(address, bytes, planes, plane stride, page stride, page bytes) of a pool [planes, pages, ...]."""
    _on_gpu(pool, "pool", contiguous=False)
    if pool.dim() < 3 or not pool[0, 0].is_contiguous():
        raise ValueError("pool must be [planes, pages, ...] with contiguous pages")
    es = pool.element_size()
    page = pool[0, 0].numel() * es
    planes, pages = pool.shape[:2]
    return (pool.data_ptr(), _span(pool) * es, planes, pool.stride(0) * es if planes > 1 else 0,
            pool.stride(1) * es if pages > 1 else page, page)


def _cache_ws(ws, n_seq, n_pages, device):
    return ws if ws is not None else decode_workspace(KIND_CACHE, n_seq, n_pages, device=device)


def lossk_cache_fork(parent, table, lens, ref, page_size, table_out=None, lens_out=None, ws=None, stream=None):
    """parent int32 [groups, n_dst]; table holds groups * n_src rows.  Returns (table_out, lens_out)."""
    _ints(parent=parent, lens=lens, ref=ref, lens_out=lens_out)
    n, m, stride = _table(table)
    G, n_dst = parent.shape
    if n % G or lens.numel() != n:
        raise ValueError(f"{n} rows and {lens.numel()} lengths in {G} groups")
    if table_out is None:
        table_out = torch.empty((G * n_dst, m), dtype=torch.int32, device=table.device)
    if lens_out is None:
        lens_out = torch.empty(G * n_dst, dtype=torch.int32, device=table.device)
    no, mo, stride_out = _table(table_out, "table_out")
    if no != G * n_dst or mo != m:
        raise ValueError("table_out must be [groups * n_dst, max_pages]")
    ws = _cache_ws(ws, max(n, no), ref.numel(), table.device)
    st = lib.lossk_cache_fork(G, n // G, n_dst, m, page_size, ref.numel(), parent.data_ptr(), parent.numel(),
                              table.data_ptr(), _span(table), stride, lens.data_ptr(), n, ref.data_ptr(), ref.numel(),
                              table_out.data_ptr(), _span(table_out), stride_out, lens_out.data_ptr(),
                              lens_out.numel(), ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "lossk_cache_fork")
    return table_out, lens_out


def lossk_cache_reserve(table, lens, ref, pool, page_size, n_new=1, ws=None, stream=None) -> None:
    """n_new: tokens to come for every sequence, or an int32 tensor with one count each."""
    _ints(lens=lens, ref=ref)
    n, m, stride = _table(table)
    each = n_new if isinstance(n_new, torch.Tensor) else None
    _ints(n_new=each)
    P = _pool(pool)
    if pool.shape[1] != ref.numel():
        raise ValueError(f"a pool of {pool.shape[1]} pages with {ref.numel()} counts")
    ws = _cache_ws(ws, n, ref.numel(), table.device)
    st = lib.lossk_cache_reserve(n, m, page_size, ref.numel(), 0 if each is not None else n_new, _ptr(each),
                                 _len(each), table.data_ptr(), _span(table), stride, lens.data_ptr(), lens.numel(),
                                 ref.data_ptr(), ref.numel(), *P, ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "lossk_cache_reserve")


def lossk_cache_free(table, lens, ref, page_size, drop=None, ws=None, stream=None) -> None:
    """drop: uint8 [n_seq], nonzero where the sequence goes (None: all)."""
    _ints(lens=lens, ref=ref)
    _on_gpu(drop, "drop", torch.uint8)
    n, m, stride = _table(table)
    ws = _cache_ws(ws, n, ref.numel(), table.device)
    st = lib.lossk_cache_free(n, m, page_size, ref.numel(), _ptr(drop), _len(drop), table.data_ptr(), _span(table),
                              stride, lens.data_ptr(), lens.numel(), ref.data_ptr(), ref.numel(), ws.data_ptr(),
                              ws.numel(), _stream(stream))
    _check(st, "lossk_cache_free")


def lossk_cache_compact(table, lens, ref, pool, page_size, table_out=None, ref_out=None, n_live_out=None, ws=None,
                        stream=None):
    """Returns (table_out, ref_out, n_live_out); the pool's live pages are in front then."""
    _ints(lens=lens, ref=ref, ref_out=ref_out, n_live_out=n_live_out)
    n, m, stride = _table(table)
    P = _pool(pool)
    if pool.shape[1] != ref.numel():
        raise ValueError(f"a pool of {pool.shape[1]} pages with {ref.numel()} counts")
    dev = table.device
    table_out = table_out if table_out is not None else torch.empty((n, m), dtype=torch.int32, device=dev)
    ref_out = ref_out if ref_out is not None else torch.empty_like(ref)
    n_live_out = n_live_out if n_live_out is not None else torch.empty(1, dtype=torch.int32, device=dev)
    no, mo, stride_out = _table(table_out, "table_out")
    if (no, mo) != (n, m) or n_live_out.numel() < 1:
        raise ValueError("table_out must be shaped like table, n_live_out hold one value")
    ws = _cache_ws(ws, n, ref.numel(), dev)
    st = lib.lossk_cache_compact(n, m, page_size, ref.numel(), table.data_ptr(), _span(table), stride,
                                 lens.data_ptr(), lens.numel(), ref.data_ptr(), ref.numel(), table_out.data_ptr(),
                                 _span(table_out), stride_out, ref_out.data_ptr(), ref_out.numel(),
                                 n_live_out.data_ptr(), *P, ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "lossk_cache_compact")
    return table_out, ref_out, n_live_out


def lossk_cache_copy(src, dst, pool, ws=None, stream=None) -> None:
    """Page src[i] of the pool to page dst[i], in every plane."""
    _ints(src=src, dst=dst)
    P = _pool(pool)
    if src.numel() != dst.numel():
        raise ValueError("src and dst must list as many pages")
    ws = ws if ws is not None else torch.zeros(256, dtype=torch.uint8, device=pool.device)
    st = lib.lossk_cache_copy(src.numel(), pool.shape[1], src.data_ptr(), src.numel(), dst.data_ptr(), dst.numel(),
                              *P, ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "lossk_cache_copy")


def _pages(k, v):
    """(pages, page size, heads, head dim, strides) of one layer's key and value pages
    [pages, page, heads, head_dim], whose elements of a head are contiguous."""
    _on_gpu(k, "k_pages", contiguous=False)
    _on_gpu(v, "v_pages", k.dtype, contiguous=False)
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or (k.shape[3] > 1 and k.stride(3) != 1):
        raise ValueError("k_pages and v_pages must be [pages, page, heads, head_dim], laid out alike, heads contiguous")
    return k.shape, k.stride()


def lossk_cache_write(k_new, v_new, k_pages, v_pages, table, lens, first=None, ws=None, stream=None) -> None:
    """k_new, v_new [n_tok, heads, head_dim] (tokens may be strided) into one layer's pages
    [pages, page, heads, head_dim] (any strides).  first: int32 [n_seq + 1], where each sequence's
    rows begin (None: one row per sequence)."""
    (n_pages, page, kv, hd), (sp, stok, sh, _) = _pages(k_pages, v_pages)
    _ints(lens=lens, first=first)
    n, m, stride = _table(table)
    for t, nm in ((k_new, "k_new"), (v_new, "v_new")):
        _on_gpu(t, nm, k_pages.dtype, contiguous=False)
        if t.dim() != 3 or t.shape[1:] != (kv, hd) or (t.shape[0] and not t[0].is_contiguous()):
            raise ValueError(f"{nm} must be [n_tok, heads, head_dim] with contiguous tokens")
    if k_new.shape != v_new.shape or k_new.stride() != v_new.stride():
        raise ValueError("k_new and v_new must be laid out alike")
    n_tok = k_new.shape[0]
    ws = ws if ws is not None else torch.zeros(256, dtype=torch.uint8, device=table.device)
    st = lib.lossk_cache_write(n_tok, n, kv, hd, m, page, n_pages, _dtype_code(k_pages), k_new.data_ptr(),
                               v_new.data_ptr(), _span(k_new), k_new.stride(0) if n_tok > 1 else kv * hd,
                               k_pages.data_ptr(), v_pages.data_ptr(), _span(k_pages), sp, stok, sh,
                               table.data_ptr(), _span(table), stride, lens.data_ptr(), lens.numel(), _ptr(first),
                               _len(first), ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "lossk_cache_write")


# ---- attention of one new token ------------------------------------------------------------

def lossk_paged_attn(q, k_pages, v_pages, table, lens, scale=None, window=0, share=1, max_len=0, out=None,
                     lse_out=None, ws=None, stream=None):
    """q [n_seq, n_q_heads, head_dim] (sequences may be strided) over one layer's pages
    [pages, page, heads, head_dim] (any strides).  scale defaults to head_dim ** -0.5; share: how
    many consecutive sequences may share leading pages.  Returns out."""
    (n_pages, page, kv, hd), (sp, stok, sh, _) = _pages(k_pages, v_pages)
    _ints(lens=lens)
    _on_gpu(q, "q", k_pages.dtype, contiguous=False)
    n, m, stride = _table(table)
    if q.dim() != 3 or q.shape[0] != n or q.shape[2] != hd or (n and not q[0].is_contiguous()):
        raise ValueError("q must be [n_seq, n_q_heads, head_dim] with contiguous sequences")
    hq = q.shape[1]
    if out is None:
        out = torch.empty((n, hq, hd), dtype=q.dtype, device=q.device)
    _on_gpu(out, "out", q.dtype)
    _on_gpu(lse_out, "lse_out", torch.float32)
    if lse_out is not None and lse_out.numel() != n * hq:
        raise ValueError("lse_out must be [n_seq, n_q_heads]")
    if ws is None:
        ws = decode_workspace(KIND_PAGED_ATTN, n, hq, kv, hd, q.device)
    st = lib.lossk_paged_attn(n, hq, kv, hd, m, page, n_pages, share, _dtype_code(q), q.data_ptr(), _span(q),
                              q.stride(0) if n > 1 else hq * hd, k_pages.data_ptr(), v_pages.data_ptr(),
                              _span(k_pages), sp, stok, sh, table.data_ptr(), _span(table), stride, lens.data_ptr(),
                              lens.numel(), max_len, window, hd ** -0.5 if scale is None else scale, out.data_ptr(),
                              out.numel(), _ptr(lse_out), ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "lossk_paged_attn")
    return out
