"""Plain 64-bit definitions of the decoding calls, for their tests (numpy, one loop per thing)."""
import math

import numpy as np


def allowed_bits(allow, V):
    """bool[rows][V] of int32 mask words [rows][ceil(V / 32)]."""
    w = np.ascontiguousarray(allow).view(np.uint32)
    v = np.arange(V)
    return ((w[:, v // 32] >> (v % 32).astype(np.uint32)) & 1).astype(bool)


def beam_select(logits, scores, n_out, temperature=1.0, allow=None, finished=None, end_token=-1, lengths=None,
                length_alpha=0.0):
    """logits float64 [B*K][V], scores [B][K]; allow bool[B*K][V] or None."""
    B, K = scores.shape
    V = logits.shape[1]
    out = {"parent": np.full((B, n_out), -1, np.int64), "token": np.full((B, n_out), -1, np.int64),
           "score": np.full((B, n_out), -np.inf), "finished": np.zeros((B, n_out), np.int64),
           "length": np.zeros((B, n_out), np.int64), "lse": np.full(B * K, -np.inf)}
    for b in range(B):
        cands = []                                     # (-rank, beam, token, score, finished, len)
        for k in range(K):
            r = b * K + k
            start = float(scores[b, k])
            done = finished is not None and bool(finished[b, k])
            ln = (0 if lengths is None else int(lengths[b, k])) + (0 if done else 1)
            div = max(1, ln) ** length_alpha
            if not math.isfinite(start):
                continue
            if done:
                cands.append((-start / div, k, end_token, start, 1, ln))
                continue
            keep = np.ones(V, bool) if allow is None else allow[r]
            x = np.where(keep, logits[r], -np.inf)
            if np.isnan(x).any() or np.isposinf(x).any() or not np.isfinite(x).any():
                continue
            x = x / temperature
            m = x.max()
            lse = m + math.log(np.exp(x - m).sum())
            out["lse"][r] = lse
            s = start + (x - lse)
            best = np.lexsort((np.arange(V), -s))[:n_out]
            cands += [(-s[v] / div, k, int(v), s[v], int(v == end_token), ln) for v in best if x[v] > -np.inf]
        cands.sort(key=lambda c: c[:3])
        for j, c in enumerate(cands[:n_out]):
            out["parent"][b, j], out["token"][b, j], out["score"][b, j] = c[1], c[2], c[3]
            out["finished"][b, j], out["length"][b, j] = c[4], c[5]
    return out
