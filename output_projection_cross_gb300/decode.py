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
           "lossk_decode_workspace_bytes", "lossk_beam_select", "lossk_beam_gather"]


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
