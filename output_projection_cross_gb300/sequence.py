"""Python binding of the losses of sampled and compared sequences: same names as the C ABI, argument marshalling only.

The clipped policy loss with a KL term and the preference loss over paired log
ratios, each from hidden rows and the head's weight or from given logits.  As in
lossk.py, every function takes torch tensors on the GPU, makes the outputs that
are left as ``None``, calls the C entry point on the current CUDA stream (or
``stream``) and raises :class:`LosskError` for any status other than 580.  Like the
decoding calls these do not synchronise: targets and ``first`` are checked on the
device, and what was found wrong there is read with ``lossk_device_status(ws)``.  So
a training loop keeps a workspace (:func:`sequence_workspace`) and passes it in.
All of a call's tensors have to be contiguous and on the current device
(``ValueError`` otherwise).
"""
from __future__ import annotations

import torch

from .decode import _calls, _NotBuilt, _on_gpu, _raw_stream, _stream_of
from .lossk import (ACCUMULATE_GRADS, F32, LosskError, _check, _contig, _dtype_code, _on_its_stream, _stream, lib,
                    lossk_dims_check)

KIND_SEQUENCE_HEAD, KIND_SEQUENCE_LOGITS = 0, 1
SEQ_RATIO, SEQ_MEAN, SEQ_ADVANTAGES, LENGTH_MEAN = 4, 8, 16, 32
OBJECTIVES = {"sigmoid": 0, "hinge": 1, "squared": 2}

__all__ = ["KIND_SEQUENCE_HEAD", "KIND_SEQUENCE_LOGITS", "SEQ_RATIO", "SEQ_MEAN", "SEQ_ADVANTAGES", "LENGTH_MEAN",
           "sequence_workspace", "lossk_sequence_workspace_bytes", "lossk_policy_fwd_bwd", "lossk_policy_from_logits",
           "lossk_preference_fwd_bwd", "lossk_preference_from_logits"]

# through the CPython module where there is one (ctypes takes 3 us for the arguments of one such call)
_lib = lib if isinstance(_calls, _NotBuilt) else _calls

# the tensors of one type that a call looks at together
_HEAD, _HEAD_GRADS, _LOGITS, _LOGITS_GRADS = ("hidden", "weight"), ("d_hidden", "d_weight"), ("logits",), ("grad_logits",)
_POLICY = ("advantages", "old_logp", "ref_logp", "scalars_out", "per_token_out", "logp_out")
_PREFERENCE = ("ref_logp", "scalars_out", "per_pair_out", "log_ratio_out", "logp_out")


def lossk_sequence_workspace_bytes(kind: int, n_tok: int, d_model: int, vocab: int, n_seq: int, dtype: int) -> int:
    return lib.lossk_sequence_workspace_bytes(kind, n_tok, d_model, vocab, n_seq, dtype)


def sequence_workspace(kind: int, n_tok: int, d_model: int, vocab: int, n_seq: int, dtype: int, device=None):
    """A zeroed workspace for calls of these sizes (n_seq: sequences, two per pair; 0 without any)."""
    nb = lib.lossk_sequence_workspace_bytes(kind, n_tok, d_model, vocab, n_seq, dtype)
    if nb < 0:
        status = lossk_dims_check(n_tok, d_model if kind == KIND_SEQUENCE_HEAD else 1, vocab)
        raise LosskError(status if status != 580 else 582, "lossk_sequence_workspace_bytes")
    return torch.zeros(nb, dtype=torch.uint8, device=device or "cuda")


def _spans(dtype, names, *tensors):
    """(address, elements) of each contiguous tensor of that type (None: any), flat; a tensor left out is 0, 0."""
    if dtype is not None and not isinstance(_calls, _NotBuilt):
        r = _calls.spans(dtype, *tensors)
        if r is not None:
            return r
    out = []
    for name, t in zip(names, tensors):
        if isinstance(_calls, _NotBuilt) and t is not None:
            _contig(t, name)
        _on_gpu(t, name, dtype)                   # (whether it is on the GPU is _handle's to say)
        out += (0, 0) if t is None else (t.data_ptr(), t.numel())
    return out


def _handle(stream, *tensors):
    """The stream's handle, once all tensors are on the current device."""
    return _stream(stream) if isinstance(_calls, _NotBuilt) else _stream_of(stream, *tensors)


def _holds(spans, *wanted):
    """wanted: (position among the spans, name, elements that it must hold unless it is left out)."""
    for i, name, n in wanted:
        if spans[2 * i] and spans[2 * i + 1] < n:
            raise ValueError(f"{name} must hold {n} elements")


def _new(t, n, device):
    return t if t is not None else torch.empty(n, dtype=torch.float32, device=device)


def _grad_type(hidden, grad_dtype, d_hidden, d_weight, want_d_hidden, want_d_weight):
    """The gradients' type: as asked for, or that of those passed in, or float."""
    types = {t.dtype for t in (d_hidden if want_d_hidden else None, d_weight if want_d_weight else None) if t is not None}
    if grad_dtype is not None:
        types.add(grad_dtype)
    if len(types) > 1:
        raise TypeError(f"d_hidden and d_weight must be of one type, not {', '.join(sorted(map(str, types)))}")
    return types.pop() if types else torch.float32


def _head(hidden, weight):
    if hidden.dim() != 2 or weight.dim() != 2 or hidden.shape[1] != weight.shape[1] or hidden.dtype != weight.dtype:
        raise ValueError("hidden must be [n_tok, d_model] and weight [vocab, d_model], of one type")
    return hidden.shape[0], hidden.shape[1], weight.shape[0], _dtype_code(hidden)


def _head_grads(hidden, weight, flags, grad_dtype, d_hidden, d_weight, want_d_hidden, want_d_weight):
    dtype = _grad_type(hidden, grad_dtype, d_hidden, d_weight, want_d_hidden, want_d_weight)
    make = torch.zeros if flags & ACCUMULATE_GRADS else torch.empty
    out = []
    for like, t, want, name in ((hidden, d_hidden, want_d_hidden, "d_hidden"), (weight, d_weight, want_d_weight, "d_weight")):
        if want and t is None:
            t = make(like.shape, dtype=dtype, device=like.device)
        if want and t.shape != like.shape:
            raise ValueError(f"{name} must be of shape {tuple(like.shape)}")
        out.append(t if want else None)
    return out[0], out[1], dtype


def _dtype_code_of(dtype):
    return F32 if dtype == torch.float32 else 1 if dtype == torch.bfloat16 else 2 if dtype == torch.float16 else -1


def _logits_grad(logits, flags, grad_logits, want_grad):
    if not want_grad:
        return None
    if grad_logits is None:
        return torch.zeros_like(logits) if flags & ACCUMULATE_GRADS else torch.empty_like(logits)
    if grad_logits.shape != logits.shape:
        raise ValueError(f"grad_logits must be of shape {tuple(logits.shape)}")
    return grad_logits


def _no_stream(f):
    """_on_its_stream without building a stream object where none is given and the raw handle is at hand."""
    on_stream = _on_its_stream(f)
    if _raw_stream is None:
        return on_stream

    def call(*args, stream=None, **kw):
        return f(*args, **kw) if stream is None else on_stream(*args, stream=stream, **kw)
    call.__name__, call.__doc__, call.__wrapped__ = f.__name__, f.__doc__, f
    return call


# ---- the policy loss ------------------------------------------------------------------

def _policy(fn, name, given, names, sizes, kind, targets, advantages, old_logp, ref_logp, first, loss_mask, scalars, flags,
            scalars_out, per_token_out, logp_out, grads, grad_names, grad_dtype, ws, stream):
    """sizes: n_tok, d_model, vocab, type; given: what the logits come from; grads: what takes their gradient."""
    n, d, V, dt = sizes
    dev = targets.device
    scalars_out, per_token_out, logp_out = _new(scalars_out, 4, dev), _new(per_token_out, n, dev), _new(logp_out, n, dev)
    n_seq = first.numel() - 1 if first is not None else 0
    if ws is None:
        ws = sequence_workspace(kind, n, d, V, max(n_seq, 0), dt, dev)
    x = _spans(given[0].dtype, names, *given)
    y = _spans(torch.int64, ("targets",), targets)
    f = _spans(torch.float32, _POLICY, advantages, old_logp, ref_logp, scalars_out, per_token_out, logp_out)
    s = _spans(torch.int32, ("first",), first)
    b = _spans(torch.uint8, ("loss_mask", "ws"), loss_mask, ws)
    g = _spans(grad_dtype, grad_names, *grads)
    _holds(y, (0, "targets", n))
    _holds(b, (0, "loss_mask", n))
    _holds(f, (3, "scalars_out", 4), (4, "per_token_out", n), (5, "logp_out", n))
    handle = _handle(stream, *given, targets, advantages, old_logp, ref_logp, scalars_out, per_token_out, logp_out, first,
                     loss_mask, ws, *grads)
    head = kind == KIND_SEQUENCE_HEAD
    _check(fn(*((n, d, V, n_seq, dt) if head else (n, V, n_seq, dt)), *x, *y, b[0], *s, *f[:6], *scalars, flags, f[6], f[8],
              f[10], *((_dtype_code_of(grad_dtype), g[0], g[2]) if head else g), b[2], b[3], handle), name)
    return {"scalars": scalars_out, "per_token": per_token_out, "logp": logp_out}


@_no_stream
def lossk_policy_fwd_bwd(hidden, weight, targets, advantages, old_logp=None, ref_logp=None, first=None, loss_mask=None,
                         clip_low=0.2, clip_high=0.2, kl_weight=0.0, temperature=1.0, grad_scale=1.0, flags=0,
                         grad_dtype=None, scalars_out=None, per_token_out=None, logp_out=None, d_hidden=None,
                         d_weight=None, want_d_hidden=True, want_d_weight=True, ws=None, stream=None) -> dict:
    """The clipped policy loss with a KL term of hidden [n_tok, d_model] and weight [vocab, d_model].

    first: int32 [n_seq + 1], or None without sequences; loss_mask: uint8 [n_tok].  advantages: float [n_tok], or
    [n_seq] with SEQ_ADVANTAGES.  grad_dtype: torch.float32 (the default), or the inputs' type.  flags:
    ACCUMULATE_GRADS, REDUCE_SUM, SEQ_RATIO, SEQ_MEAN, SEQ_ADVANTAGES.  With want_d_hidden and want_d_weight
    False it is the forward pass alone (the log-probabilities of a sampling policy or a reference model).
    Returns scalars (total, policy, KL, clipped share), per_token, logp, d_hidden, d_weight."""
    n, d, V, dt = _head(hidden, weight)
    d_hidden, d_weight, grad_dtype = _head_grads(hidden, weight, flags, grad_dtype, d_hidden, d_weight, want_d_hidden,
                                                 want_d_weight)
    out = _policy(_lib.lossk_policy_fwd_bwd, "lossk_policy_fwd_bwd", (hidden, weight), _HEAD, (n, d, V, dt),
                  KIND_SEQUENCE_HEAD, targets, advantages, old_logp, ref_logp, first, loss_mask,
                  (clip_low, clip_high, kl_weight, temperature, grad_scale), flags, scalars_out, per_token_out, logp_out,
                  (d_hidden, d_weight), _HEAD_GRADS, grad_dtype, ws, stream)
    out["d_hidden"], out["d_weight"] = d_hidden, d_weight
    return out


@_no_stream
def lossk_policy_from_logits(logits, targets, advantages, old_logp=None, ref_logp=None, first=None, loss_mask=None,
                             clip_low=0.2, clip_high=0.2, kl_weight=0.0, temperature=1.0, grad_scale=1.0, flags=0,
                             want_grad=True, scalars_out=None, per_token_out=None, logp_out=None, grad_logits=None,
                             ws=None, stream=None) -> dict:
    """The same of logits [n_tok, vocab]; returns grad_logits (the logits' type) instead of d_hidden and d_weight."""
    n, V = logits.shape
    dt = _dtype_code(logits)
    grad_logits = _logits_grad(logits, flags, grad_logits, want_grad)
    out = _policy(_lib.lossk_policy_from_logits, "lossk_policy_from_logits", (logits,), _LOGITS, (n, 1, V, dt),
                  KIND_SEQUENCE_LOGITS, targets, advantages, old_logp, ref_logp, first, loss_mask,
                  (clip_low, clip_high, kl_weight, temperature, grad_scale), flags, scalars_out, per_token_out, logp_out,
                  (grad_logits,), _LOGITS_GRADS, logits.dtype, ws, stream)
    out["grad_logits"] = grad_logits
    return out


# ---- the preference loss ----------------------------------------------------------------

def _preference(fn, name, given, names, sizes, kind, targets, first, ref_logp, loss_mask, objective, scalars, flags,
                scalars_out, per_pair_out, log_ratio_out, logp_out, grads, grad_names, grad_dtype, ws, stream):
    n, d, V, dt = sizes
    dev = targets.device
    if first.numel() % 2 != 1:
        raise ValueError("first must hold 2 * n_pairs + 1 elements")
    pairs = first.numel() // 2
    scalars_out, per_pair_out = _new(scalars_out, 4, dev), _new(per_pair_out, pairs, dev)
    log_ratio_out, logp_out = _new(log_ratio_out, 2 * pairs, dev), _new(logp_out, n, dev)
    if ws is None:
        ws = sequence_workspace(kind, n, d, V, 2 * pairs, dt, dev)
    x = _spans(given[0].dtype, names, *given)
    y = _spans(torch.int64, ("targets",), targets)
    f = _spans(torch.float32, _PREFERENCE, ref_logp, scalars_out, per_pair_out, log_ratio_out, logp_out)
    s = _spans(torch.int32, ("first",), first)
    b = _spans(torch.uint8, ("loss_mask", "ws"), loss_mask, ws)
    g = _spans(grad_dtype, grad_names, *grads)
    _holds(y, (0, "targets", n))
    _holds(b, (0, "loss_mask", n))
    _holds(f, (1, "scalars_out", 4), (2, "per_pair_out", pairs), (3, "log_ratio_out", 2 * pairs), (4, "logp_out", n))
    handle = _handle(stream, *given, targets, first, ref_logp, scalars_out, per_pair_out, log_ratio_out, logp_out, loss_mask,
                     ws, *grads)
    head = kind == KIND_SEQUENCE_HEAD
    _check(fn(*((n, d, V, pairs, dt) if head else (n, V, pairs, dt)), *x, *y, b[0], *s, f[0], f[1],
              OBJECTIVES[objective] if isinstance(objective, str) else int(objective), *scalars, flags, f[2], f[4], f[6],
              f[8], *((_dtype_code_of(grad_dtype), g[0], g[2]) if head else g), b[2], b[3], handle), name)
    return {"scalars": scalars_out, "per_pair": per_pair_out, "log_ratio": log_ratio_out, "logp": logp_out}


@_no_stream
def lossk_preference_fwd_bwd(hidden, weight, targets, first, ref_logp=None, loss_mask=None, objective="sigmoid", beta=0.1,
                             margin=0.0, label_smoothing=0.0, nll_weight=0.0, grad_scale=1.0, flags=0, grad_dtype=None,
                             scalars_out=None, per_pair_out=None, log_ratio_out=None, logp_out=None, d_hidden=None,
                             d_weight=None, want_d_hidden=True, want_d_weight=True, ws=None, stream=None) -> dict:
    """The preference loss of hidden [n_tok, d_model] and weight [vocab, d_model].

    first: int32 [2 * n_pairs + 1], the chosen sequences and then the rejected ones; ref_logp: float [n_tok], the
    reference model's log-probabilities, or None.  objective: "sigmoid", "hinge" or "squared".  flags:
    ACCUMULATE_GRADS, REDUCE_SUM, LENGTH_MEAN.  Returns scalars (total, preference, -logp of the chosen tokens,
    share of pairs in order), per_pair, log_ratio (per sequence), logp, d_hidden, d_weight."""
    n, d, V, dt = _head(hidden, weight)
    d_hidden, d_weight, grad_dtype = _head_grads(hidden, weight, flags, grad_dtype, d_hidden, d_weight, want_d_hidden,
                                                 want_d_weight)
    out = _preference(_lib.lossk_preference_fwd_bwd, "lossk_preference_fwd_bwd", (hidden, weight), _HEAD, (n, d, V, dt),
                      KIND_SEQUENCE_HEAD, targets, first, ref_logp, loss_mask, objective,
                      (beta, margin, label_smoothing, nll_weight, grad_scale), flags, scalars_out, per_pair_out,
                      log_ratio_out, logp_out, (d_hidden, d_weight), _HEAD_GRADS, grad_dtype, ws, stream)
    out["d_hidden"], out["d_weight"] = d_hidden, d_weight
    return out


@_no_stream
def lossk_preference_from_logits(logits, targets, first, ref_logp=None, loss_mask=None, objective="sigmoid", beta=0.1,
                                 margin=0.0, label_smoothing=0.0, nll_weight=0.0, grad_scale=1.0, flags=0,
                                 want_grad=True, scalars_out=None, per_pair_out=None, log_ratio_out=None, logp_out=None,
                                 grad_logits=None, ws=None, stream=None) -> dict:
    """The same of logits [n_tok, vocab]; returns grad_logits (the logits' type) instead of d_hidden and d_weight."""
    n, V = logits.shape
    dt = _dtype_code(logits)
    grad_logits = _logits_grad(logits, flags, grad_logits, want_grad)
    out = _preference(_lib.lossk_preference_from_logits, "lossk_preference_from_logits", (logits,), _LOGITS, (n, 1, V, dt),
                      KIND_SEQUENCE_LOGITS, targets, first, ref_logp, loss_mask, objective,
                      (beta, margin, label_smoothing, nll_weight, grad_scale), flags, scalars_out, per_pair_out,
                      log_ratio_out, logp_out, (grad_logits,), _LOGITS_GRADS, logits.dtype, ws, stream)
    out["grad_logits"] = grad_logits
    return out
