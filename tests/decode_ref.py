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


class Cache:
    """A paged cache kept by hand: tables as lists of pages, the pool as an array [planes][pages][page][row]."""

    def __init__(self, pool, page, rows):
        self.pool, self.page = pool.copy(), page
        self.rows, self.lens = [list(r) for r in rows], [0] * len(rows)

    def ref(self):
        n = np.zeros(self.pool.shape[1], np.int64)
        for r in self.rows:
            for p in r:
                n[p] += 1
        return n

    def table(self, max_pages):
        t = np.full((len(self.rows), max_pages), -1, np.int32)
        for i, r in enumerate(self.rows):
            t[i, :len(r)] = r
        return t

    def used(self, i):
        return -(-self.lens[i] // self.page)

    def fork(self, parent, n_src):
        take = [None if p < 0 else g * n_src + p for g, ps in enumerate(parent) for p in ps]
        self.rows = [[] if s is None else list(self.rows[s][:self.used(s)]) for s in take]
        self.lens = [0 if s is None else self.lens[s] for s in take]

    def reserve(self, n_new):
        """False, with nothing changed, where there are too few free pages."""
        ref = self.ref()
        free = [p for p in range(len(ref)) if ref[p] == 0]
        copies = []
        for i, r in enumerate(self.rows):
            if n_new[i] and self.lens[i] % self.page:
                p = r[self.lens[i] // self.page]
                who = [j for j, q in enumerate(self.rows) if n_new[j] and self.lens[j] % self.page
                       and q[self.lens[j] // self.page] == p]
                if not (ref[p] == len(who) and i == who[-1]):
                    copies.append(i)
        add = [-(-(self.lens[i] + n_new[i]) // self.page) - self.used(i) for i in range(len(self.rows))]
        if len(copies) + sum(add) > len(free):
            return False
        for i, r in enumerate(self.rows):
            if i in copies:
                c = self.lens[i] // self.page
                self.pool[:, free[0]] = self.pool[:, r[c]]
                r[c] = free.pop(0)
            for _ in range(add[i]):
                r.append(free.pop(0))
        return True

    def write(self, k_new, v_new, first):
        for i, r in enumerate(self.rows):
            for j in range(first[i], first[i + 1]):
                pos = self.lens[i] + j - first[i]
                self.pool[0, r[pos // self.page], pos % self.page] = k_new[j]
                self.pool[1, r[pos // self.page], pos % self.page] = v_new[j]

    def free(self, drop):
        for i, d in enumerate(drop):
            if d:
                self.rows[i], self.lens[i] = [], 0

    def compact(self):
        ref = self.ref()
        n = int((ref > 0).sum())
        to = dict(zip([p for p in range(n, len(ref)) if ref[p]], [p for p in range(n) if not ref[p]]))
        for a, b in to.items():
            self.pool[:, b] = self.pool[:, a]
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        return n


def attend(q, k, v, table, lens, page, scale, window=0):
    """q [S][Hq][hd], k and v [pages][page][Hkv][hd], all float64.  Returns (out, lse)."""
    S, Hq, hd = q.shape
    group = Hq // k.shape[2]
    out, lse = np.zeros((S, Hq, hd)), np.full((S, Hq), -np.inf)
    for s in range(S):
        n = int(lens[s])
        j = np.arange(max(0, n - window) if window else 0, n)
        if not len(j):
            continue
        kk, vv = k[table[s, j // page], j % page], v[table[s, j // page], j % page]
        for h in range(Hq):
            x = kk[:, h // group] @ q[s, h] * scale
            m = x.max()
            p = np.exp(x - m)
            out[s, h], lse[s, h] = p @ vv[:, h // group] / p.sum(), m + math.log(p.sum())
    return out, lse
