"""The operators of beam-search decoding, each as one measured pass.

Four kinds of pass, over one vocabulary head and one paged key-value cache:

  select   beam selection over beams and vocabulary (lossk_beam_select)
  attend   attention of one new token per sequence over the paged cache
           (lossk_paged_attn)
  step     the cache's side of one decoding step: fork the sequences by their
           parents, reserve a slot for the next token (allocating pages and
           copying shared partial ones), write the new token's rows
           (lossk_cache_fork, lossk_cache_reserve, lossk_cache_write)
  compact  live pages moved to the front of the pool (lossk_cache_compact)

With ``own`` false a pass runs the operator's plain form in elementary torch
operations; with ``own`` true it calls the package.  ``exact`` is the
definition in 64 bits, written apart from the plain form.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # One interactive request with four beams and a mid-sized vocabulary: all latency.
        {"name": "select 1x4, 32000, bf16", "op": "select", "batch": 1, "beams": 4, "vocab": 32000, "dtype": "bf16",
         "n_out": 8, "temperature": 1.0, "allow": "none", "finished": 0.0, "alpha": 0.0},
        # An odd vocabulary with fp32 logits, a grammar's bit mask per beam, some beams finished
        # and length-normalised ranks.
        {"name": "select 5x7, 32003, f32, masked", "op": "select", "batch": 5, "beams": 7, "vocab": 32003,
         "dtype": "f32", "n_out": 14, "temperature": 0.7, "allow": "row", "finished": 0.25, "alpha": 0.6},
        # A small serving batch at a large vocabulary: 64 rows of logits.
        {"name": "select 16x4, 151936, bf16", "op": "select", "batch": 16, "beams": 4, "vocab": 151936,
         "dtype": "bf16", "n_out": 8, "temperature": 1.0, "allow": "none", "finished": 0.0, "alpha": 0.0},
        # Sequence-level distillation decoding a whole batch of prompts: 311 MB of logits.
        {"name": "select 128x8, 151936, bf16", "op": "select", "batch": 128, "beams": 8, "vocab": 151936,
         "dtype": "bf16", "n_out": 16, "temperature": 1.0, "allow": "none", "finished": 0.1, "alpha": 1.0},
        # One interactive request: 512 cached tokens, all latency.
        {"name": "attend 1 seq, 512 tokens, bf16", "op": "attend", "groups": 1, "share": 1, "prefix": 0, "min_len": 512,
         "max_len": 512, "hq": 16, "hkv": 8, "hd": 128, "page": 16, "layout": "token", "window": 0, "dtype": "bf16"},
        # Continuous batching: ragged lengths from one token to 9000.
        {"name": "attend 33 seqs, 1..9000 tokens, f16", "op": "attend", "groups": 33, "share": 1, "prefix": 0,
         "min_len": 1, "max_len": 9000, "hq": 32, "hkv": 8, "hd": 128, "page": 16, "layout": "head", "window": 0,
         "dtype": "f16"},
        # Beam search: 8 prompts of 4096 tokens, 8 beams each that share the prompt's pages.
        {"name": "attend 8x8 beams, 4096 shared, bf16", "op": "attend", "groups": 8, "share": 8, "prefix": 4096,
         "min_len": 4106, "max_len": 4350, "hq": 32, "hkv": 8, "hd": 128, "page": 32, "layout": "token", "window": 0,
         "dtype": "bf16"},
        # One very long document: 131072 cached tokens.
        {"name": "attend 1 seq, 131072 tokens, bf16", "op": "attend", "groups": 1, "share": 1, "prefix": 0,
         "min_len": 131072, "max_len": 131072, "hq": 32, "hkv": 8, "hd": 128, "page": 64, "layout": "token",
         "window": 0, "dtype": "bf16"},
        # One request's four beams advance by a token.
        {"name": "step 1x4 beams, 300 tokens", "op": "step", "groups": 1, "beams": 4, "len": 300, "planes": 4, "hkv": 8,
         "hd": 128, "page": 16, "pages": 160, "dtype": "bf16"},
        # A large batch of beams advances by a token.
        {"name": "step 64x8 beams, 1501 tokens", "op": "step", "groups": 64, "beams": 8, "len": 1501, "planes": 4,
         "hkv": 8, "hd": 128, "page": 16, "pages": 13312, "dtype": "bf16"},
        # A small pool tidied between requests; odd page and pool sizes.
        {"name": "compact 331 pages", "op": "compact", "seqs": 9, "planes": 6, "hkv": 2, "hd": 64, "page": 24,
         "pages": 331, "live": 0.45, "shared": 0.2, "dtype": "f16"},
        # A fragmented pool tidied so that its tail can be given back.
        {"name": "compact 8192 pages", "op": "compact", "seqs": 96, "planes": 4, "hkv": 8, "hd": 128, "page": 16,
         "pages": 8192, "live": 0.6, "shared": 0.3, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["select", "select", "attend", "attend", "attend", "step", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "select":
        vocab = _log_int(rng, 1, 151936)
        beams = rng.randint(1, 16)
        batch = _log_int(rng, 1, 128)
        while batch * beams * vocab * ESIZE[dtype] > 300e6 and batch > 1:
            batch //= 2
        return {"op": op, "batch": batch, "beams": beams, "vocab": vocab, "dtype": dtype,
                "n_out": rng.randint(1, 2 * beams), "temperature": rng.choice([1.0, rng.uniform(0.3, 2.0)]),
                "allow": rng.choice(["none", "none", "row", "all"]), "finished": rng.choice([0.0, rng.uniform(0.0, 0.6)]),
                "alpha": rng.choice([0.0, 1.0, rng.uniform(0.2, 1.2)])}
    if op == "attend":
        hkv = rng.randint(1, 12)
        hd = 8 * rng.randint(4, 32)
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        share = rng.choice([1, 1, 2, rng.randint(3, 10)])
        groups = _log_int(rng, 1, 48)
        token_bytes = hkv * hd * 2 * ESIZE[dtype]
        cap = max(16, min(131072, int(400e6 / (token_bytes * groups * share))))
        max_len = _log_int(rng, 1, cap)
        min_len = rng.choice([max_len, _log_int(rng, 1, max_len), 0])
        prefix = 0 if share == 1 else rng.randint(0, min_len)
        return {"op": op, "groups": groups, "share": share, "prefix": prefix, "min_len": min_len, "max_len": max_len,
                "hq": hkv * group, "hkv": hkv, "hd": hd, "page": rng.choice([1, 8, 16, 16, 20, 32, 64, 128, 256]),
                "layout": rng.choice(["token", "head"]), "window": rng.choice([0, 0, rng.randint(1, max_len)]),
                "dtype": dtype}
    hkv, hd, page = rng.randint(1, 8), 8 * rng.randint(4, 16), rng.choice([8, 16, 16, 24, 32, 64])
    plane_bytes = page * hkv * hd * ESIZE[dtype]
    planes = 2 * rng.randint(1, 4)
    if op == "step":
        groups, beams = _log_int(rng, 1, 64), rng.randint(1, 12)
        length = _log_int(rng, 1, 1500)
        used = -(-length // page)
        pages = groups * (used + beams * (2 + used // 4) + beams) + rng.randint(1, 64)
        while pages * planes * plane_bytes > 1.6e9 and groups > 1:
            groups //= 2
            pages = groups * (used + beams * (2 + used // 4) + beams) + rng.randint(1, 64)
        return {"op": op, "groups": groups, "beams": beams, "len": length, "planes": planes, "hkv": hkv, "hd": hd,
                "page": page, "pages": pages, "dtype": dtype}
    pages = _log_int(rng, 4, 8192)
    while pages * planes * plane_bytes > 1.0e9:
        pages //= 2
    return {"op": op, "seqs": _log_int(rng, 1, max(1, min(96, pages // 4))), "planes": planes, "hkv": hkv, "hd": hd,
            "page": page, "pages": pages, "live": rng.uniform(0.05, 0.95), "shared": rng.uniform(0.0, 0.5),
            "dtype": dtype}


# ---- what the cases share ---------------------------------------------------------

def _gens(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return np.random.default_rng([seed, 17]), g


def _randn(gen, shape, dtype):
    return torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32).to(dtype)


def _lens(case):
    """The sequence lengths of an attend case, one per group: spread over the range's logarithm."""
    n, lo, hi = case["groups"], case["min_len"], case["max_len"]
    if n == 1:
        return [hi]
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]


def _finished_count(case):
    return int(round(case["finished"] * case["beams"])) if case["beams"] > 1 else 0


def _step_distinct(beams):
    """How many of a group's beams go on; the others are dropped for copies of these."""
    return (beams + 1) // 2


def _compact_counts(case):
    """(live pages, those of them that have to move)."""
    n = case["pages"]
    live = max(1, min(n - 1, int(round(case["live"] * n))))
    moved = int(round(live * (n - live) / n))
    return live, max(0, min(moved, live, n - live))


def work(case):
    es = ESIZE[case["dtype"]]
    if case["op"] == "select":
        rows = case["batch"] * (case["beams"] - _finished_count(case))
        masks = {"none": 0, "all": 1, "row": rows}[case["allow"]]
        b = rows * case["vocab"] * es + masks * ((case["vocab"] + 31) // 32) * 4
        b += case["batch"] * case["beams"] * 4 + case["batch"] * case["n_out"] * 16
        return {"bytes": b, "flops": 4 * rows * case["vocab"]}
    if case["op"] == "attend":
        read = seen = 0
        for n in _lens(case):
            w = min(n, case["window"]) if case["window"] else n
            seen += w * case["share"]
            shared = max(0, min(case["prefix"] // case["page"] * case["page"], n) - (n - w)) if case["share"] > 1 else 0
            read += shared + (w - shared) * case["share"]
        rows = case["groups"] * case["share"] * case["hq"]
        return {"bytes": read * case["hkv"] * case["hd"] * 2 * es + rows * (case["hd"] * 2 * es + 4),
                "flops": 4 * seen * case["hq"] * case["hd"]}
    page_bytes = case["page"] * case["hkv"] * case["hd"] * es
    if case["op"] == "step":
        seqs, used = case["groups"] * case["beams"], -(-case["len"] // case["page"])
        copies = case["groups"] * (case["beams"] - _step_distinct(case["beams"])) if case["len"] % case["page"] else 0
        rows = seqs * 2 * case["hkv"] * case["hd"] * es
        return {"bytes": copies * case["planes"] * 2 * page_bytes + 2 * rows + seqs * (2 * used * 4 + 12)
                + case["pages"] * 4, "flops": 0}
    live, moved = _compact_counts(case)
    entries = live * (1 + case["shared"])
    return {"bytes": int(moved * case["planes"] * 2 * page_bytes + entries * 8 + case["pages"] * 8), "flops": 0}


# ---- inputs -----------------------------------------------------------------------

def prepare(case, seed):
    s = {"case": case}
    globals()["_prepare_" + case["op"]](case, seed, s)
    if own:
        import output_projection_cross_gb300 as L
        s["L"] = L
        globals()["_own_" + case["op"]](case, s, L)
    return s


def _prepare_select(case, seed, s):
    rng, gen = _gens(seed)
    B, K, V = case["batch"], case["beams"], case["vocab"]
    # a next-token distribution: a few likely tokens over a wide floor, frequent tokens favoured
    x = torch.randn((B * K, V), device="cuda", generator=gen)
    x *= 2.5
    x -= 0.6 * torch.log(torch.arange(1, V + 1, device="cuda", dtype=torch.float32))
    s["logits"] = x.to(DTYPES[case["dtype"]])
    del x
    s["scores"] = -torch.rand((B, K), device="cuda", generator=gen) * 6.0 - 0.5
    s["lengths"] = torch.from_numpy(rng.integers(1, 200, (B, K)).astype(np.int32)).cuda() if case["alpha"] else None
    s["end"] = int(rng.integers(0, V))
    fin = np.zeros((B, K), np.uint8)
    for b in range(B):
        fin[b, rng.permutation(K)[:_finished_count(case)]] = 1
    s["finished"] = torch.from_numpy(fin).cuda()
    s["allow"] = None
    if case["allow"] != "none":
        words = (V + 31) // 32
        rows = 1 if case["allow"] == "all" else B * K
        # a grammar lets a part of the vocabulary through; now and then it leaves a beam nothing
        bits = rng.integers(0, 1 << 32, (rows, words), dtype=np.uint64).astype(np.uint32)
        if rows > 3:
            bits[rng.integers(0, rows)] = 0
        s["allow"] = torch.from_numpy(bits.view(np.int32)).cuda()


def _make_tables(rng, groups, share, lens, prefix_pages, page, spare, max_pages):
    """Tables of groups whose sequences share their first prefix_pages pages: (table, pages in the pool)."""
    rows = []
    nxt = 0
    for g in range(groups):
        used = -(-lens[g] // page)
        pre = min(prefix_pages, used) if share > 1 else 0
        common = list(range(nxt, nxt + pre))
        nxt += pre
        for _ in range(share):
            rows.append(common + list(range(nxt, nxt + used - pre)))
            nxt += used - pre
    n_pages = nxt + spare
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((groups * share, max_pages), -1, np.int32)
    for i, r in enumerate(rows):
        table[i, :len(r)] = perm[np.array(r, np.int64)] if r else []
    return table, n_pages


def _prepare_attend(case, seed, s):
    rng, gen = _gens(seed)
    page, hkv, hd, dt = case["page"], case["hkv"], case["hd"], DTYPES[case["dtype"]]
    lens = _lens(case)
    max_pages = max(1, -(-max(lens) // page))
    lens = [lens[i] for i in rng.permutation(len(lens))]
    table, n_pages = _make_tables(rng, case["groups"], case["share"], lens, case["prefix"] // page, page, 3, max_pages)
    s["table"] = torch.from_numpy(table).cuda()
    s["lens"] = torch.from_numpy(np.repeat(np.array(lens, np.int32), case["share"])).cuda()
    shape = (2, n_pages, page, hkv, hd) if case["layout"] == "token" else (2, n_pages, hkv, page, hd)
    kv = _randn(gen, shape, dt)
    s["k"], s["v"] = (kv[0], kv[1]) if case["layout"] == "token" else (kv[0].transpose(1, 2), kv[1].transpose(1, 2))
    s["q"] = _randn(gen, (case["groups"] * case["share"], case["hq"], hd), dt)
    s["scale"] = hd ** -0.5
    s["max_len"] = max(lens)


def _prepare_step(case, seed, s):
    rng, gen = _gens(seed)
    G, K, n, page, P = case["groups"], case["beams"], case["len"], case["page"], case["pages"]
    used = -(-n // page)
    max_pages = used + 2
    table = np.full((G * K, max_pages), -1, np.int64)
    nxt = 0
    parent = np.zeros((G, K), np.int32)
    for g in range(G):
        for k in range(K):
            r = table[g * K + k]
            # a beam shares its pages with an earlier one up to where the two parted: somewhere
            # in the last quarter, before the page that is being filled
            first = 0
            if k:
                first = int(rng.integers(max(0, used - 1 - used // 4), max(1, used)))
                r[:first] = table[g * K + int(rng.integers(0, k)), :first]
            r[first:used] = np.arange(nxt, nxt + used - first)
            nxt += used - first
        keep = rng.permutation(K)[:_step_distinct(K)]
        extra = keep[rng.integers(0, len(keep), K - len(keep))]
        parent[g] = rng.permutation(np.concatenate([keep, extra]))
    if nxt + G * K > P:
        raise ValueError("the pool of this case is too small")
    perm = rng.permutation(P)
    table = np.where(table >= 0, perm[np.maximum(table, 0)], -1).astype(np.int32)
    ref = np.bincount(table[table >= 0], minlength=P).astype(np.int32)
    s["table"] = torch.from_numpy(table).cuda()
    s["lens"] = torch.full((G * K,), n, dtype=torch.int32, device="cuda")
    s["ref0"] = torch.from_numpy(ref).cuda()
    s["ref"] = s["ref0"].clone()
    s["parent"] = torch.from_numpy(parent).cuda()
    s["pool"] = _randn(gen, (case["planes"], P, page, case["hkv"], case["hd"]), DTYPES[case["dtype"]])
    s["k_new"] = _randn(gen, (G * K, case["hkv"], case["hd"]), DTYPES[case["dtype"]])
    s["v_new"] = _randn(gen, (G * K, case["hkv"], case["hd"]), DTYPES[case["dtype"]])


def _prepare_compact(case, seed, s):
    rng, gen = _gens(seed)
    P, page, S = case["pages"], case["page"], case["seqs"]
    live, moved = _compact_counts(case)
    low, high = rng.permutation(live), live + rng.permutation(P - live)
    ids = rng.permutation(np.concatenate([low[:live - moved], high[:moved]]))
    # every live page belongs to a sequence, long and short ones; some belong to a second one as well
    share = np.cumsum(0.5 + np.arange(S) / S)
    rows = [list(r) for r in np.split(ids, (live * share / share[-1]).astype(np.int64)[:-1])]
    for i in range(int(round(case["shared"] * live)) if S > 1 else 0):
        rows[i % S].append(int(ids[rng.integers(0, live)]))
    max_pages = max(1, max(len(r) for r in rows))
    table = np.full((S, max_pages), -1, np.int32)
    lens = np.zeros(S, np.int32)
    for i, r in enumerate(rows):
        table[i, :len(r)] = r
        lens[i] = len(r) * page - (int(rng.integers(0, page)) if r else 0)
    s["table"] = torch.from_numpy(table).cuda()
    s["lens"] = torch.from_numpy(lens).cuda()
    s["ref"] = torch.from_numpy(np.bincount(table[table >= 0], minlength=P).astype(np.int32)).cuda()
    s["pool"] = _randn(gen, (case["planes"], P, page, case["hkv"], case["hd"]), DTYPES[case["dtype"]])


# ---- one pass ---------------------------------------------------------------------

def run(s):
    return globals()[("_run_own_" if own else "_run_plain_") + s["case"]["op"]](s)


# The package's calls, on buffers and a workspace that a decoding loop keeps.

def _own_select(case, s, L):
    B, K = case["batch"], case["beams"]
    s["ws"] = L.decode_workspace(L.KIND_BEAM_SELECT, B, K, case["vocab"], case["n_out"])
    s["out"] = L.beam_buffers(B, case["n_out"], "cuda")


def _run_own_select(s):
    c, o = s["case"], s["out"]
    s["L"].lossk_beam_select(s["logits"], s["scores"], c["n_out"], temperature=c["temperature"], allow=s["allow"],
                             finished=s["finished"], end_token=s["end"], lengths=s["lengths"],
                             length_alpha=c["alpha"], out=o, ws=s["ws"])
    return {"parent": o["parent"], "token": o["token"], "score": o["score"], "finished": o["finished"]}


def _own_attend(case, s, L):
    s["ws"] = L.decode_workspace(L.KIND_PAGED_ATTN, s["q"].shape[0], case["hq"], case["hkv"], case["hd"])
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")


def _run_own_attend(s):
    c = s["case"]
    s["L"].lossk_paged_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"], window=c["window"],
                            share=c["share"], max_len=s["max_len"], out=s["out"], lse_out=s["lse"], ws=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_step(case, s, L):
    s["ws"] = L.decode_workspace(L.KIND_CACHE, s["lens"].numel(), case["pages"])
    s["table_out"], s["lens_out"] = torch.empty_like(s["table"]), torch.empty_like(s["lens"])


def _run_own_step(s):
    L, c = s["L"], s["case"]
    s["ref"].copy_(s["ref0"])
    L.lossk_cache_fork(s["parent"], s["table"], s["lens"], s["ref"], c["page"], table_out=s["table_out"],
                       lens_out=s["lens_out"], ws=s["ws"])
    L.lossk_cache_reserve(s["table_out"], s["lens_out"], s["ref"], s["pool"], c["page"], ws=s["ws"])
    L.lossk_cache_write(s["k_new"], s["v_new"], s["pool"][0], s["pool"][1], s["table_out"], s["lens_out"], ws=s["ws"])
    return {"table": s["table_out"], "lens": s["lens_out"], "ref": s["ref"], "pool": s["pool"]}


def _own_compact(case, s, L):
    s["ws"] = L.decode_workspace(L.KIND_CACHE, case["seqs"], case["pages"])
    s["table_out"], s["ref_out"] = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
    s["n_live"] = torch.empty(1, dtype=torch.int32, device="cuda")


def _run_own_compact(s):
    s["L"].lossk_cache_compact(s["table"], s["lens"], s["ref"], s["pool"], s["case"]["page"],
                               table_out=s["table_out"], ref_out=s["ref_out"], n_live_out=s["n_live"], ws=s["ws"])
    return {"table": s["table_out"], "ref": s["ref_out"], "n_live": s["n_live"], "pool": s["pool"]}


# The plain forms.

def _bits(allow, V):
    return ((allow.unsqueeze(-1) >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).bool().flatten(1)[:, :V]


def _run_plain_select(s):
    c = s["case"]
    B, K, V, N, T = c["batch"], c["beams"], c["vocab"], c["n_out"], c["temperature"]
    kk = min(N, V)
    x = s["logits"].float() + 0.0
    if s["allow"] is not None:
        x = torch.where(_bits(s["allow"], V), x, torch.full((), -math.inf, device="cuda"))
    m = x.amax(-1)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    # the sum and what follows in 64 bits: beams are ranked against one another by their scores
    lse = torch.exp(((x - m[:, None]).double() / T).float()).sum(-1, dtype=torch.float64).log() + m.double() / T
    # a row's candidates by logit, the lowest index first among equals
    i = x.view(torch.int32)
    key = ((i ^ ((i >> 31) & 0x7FFFFFFF)).long() << 32) + (0x7FFFFFFF - torch.arange(V, device="cuda"))
    tok = 0x7FFFFFFF - (torch.topk(key, kk, dim=-1).values & 0xFFFFFFFF)
    xv = torch.gather(x, 1, tok)
    fin = s["finished"].bool().view(B, K)
    lens = s["lengths"] if s["lengths"] is not None else torch.zeros((B, K), dtype=torch.int32, device="cuda")
    beam = s["scores"].double()
    score = beam[:, :, None] + (xv.double() / T - lse[:, None]).view(B, K, kk)
    ok = (xv > -math.inf).view(B, K, kk) & torch.isfinite(beam)[:, :, None]
    first = (torch.arange(kk, device="cuda") == 0).expand(B, K, kk)
    tok = torch.where(fin[:, :, None], torch.full((), s["end"], device="cuda"), tok.view(B, K, kk))
    score = torch.where(fin[:, :, None], beam[:, :, None], score)
    ok = torch.where(fin[:, :, None], first & torch.isfinite(beam)[:, :, None], ok)
    new_len = lens + (~fin)
    rank = score / new_len.clamp(min=1).double().pow(c["alpha"])[:, :, None]
    rank = torch.where(ok, rank, torch.full((), -math.inf, device="cuda", dtype=torch.float64)).view(B, -1)
    par = torch.arange(K, device="cuda")[None, :, None].expand(B, K, kk).reshape(B, -1)
    tok, score, ok = tok.reshape(B, -1), score.reshape(B, -1), ok.reshape(B, -1)
    flat = torch.where(ok, par * V + tok, torch.full((), 1 << 60, device="cuda"))
    o = torch.argsort(flat, dim=-1)
    o = torch.gather(o, 1, torch.sort(torch.gather(rank, 1, o), dim=-1, descending=True, stable=True).indices)
    if o.shape[1] < N:
        pad = N - o.shape[1]
        o = torch.cat([o, torch.zeros((B, pad), dtype=torch.int64, device="cuda")], 1)
        keep = torch.arange(N, device="cuda") < N - pad
    else:
        o, keep = o[:, :N], torch.ones(N, dtype=torch.bool, device="cuda")
    ok = torch.gather(ok, 1, o) & keep
    par, tok = torch.gather(par, 1, o), torch.gather(tok, 1, o)
    done = (torch.gather(fin, 1, par) | (tok == s["end"])) & ok
    return {"parent": torch.where(ok, par, -1).int(), "token": torch.where(ok, tok, -1),
            "score": torch.where(ok, torch.gather(score, 1, o), -math.inf).float(), "finished": done.to(torch.uint8)}


def _run_plain_attend(s):
    c = s["case"]
    S, hq, hd = s["q"].shape
    hkv = c["hkv"]
    used = max(1, -(-s["max_len"] // c["page"]))
    idx = s["table"][:, :used].long().clamp(min=0)
    n = used * c["page"]
    k = s["k"][idx].float().reshape(S, n, hkv, hd).transpose(1, 2)
    v = s["v"][idx].float().reshape(S, n, hkv, hd).transpose(1, 2)
    q = s["q"].float().view(S, hkv, hq // hkv, hd)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    pos = torch.arange(n, device="cuda")
    lens = s["lens"].long()
    lo = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    seen = ((pos >= lo[:, None]) & (pos < lens[:, None]))[:, None, None, :]
    x = torch.where(seen, x, torch.full((), -math.inf, device="cuda"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    v = torch.where(seen.view(S, 1, n, 1), v, torch.zeros((), device="cuda"))
    o = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    return {"out": o.reshape(S, hq, hd).to(s["q"].dtype), "lse": (m + torch.log(z)).view(S, hq)}


def _run_plain_step(s):
    c = s["case"]
    G, K, page, P = c["groups"], c["beams"], c["page"], c["pages"]
    S = G * K
    ref = s["ref"].copy_(s["ref0"])
    # fork: each sequence takes its parent's pages; references move with them
    src = (s["parent"].long() + K * torch.arange(G, device="cuda")[:, None]).flatten()
    lens = s["lens"][src]
    cols = torch.arange(s["table"].shape[1], device="cuda")
    used = (s["lens"] + page - 1) // page
    children = torch.zeros(S, dtype=torch.int32, device="cuda").scatter_add_(
        0, src, torch.ones(S, dtype=torch.int32, device="cuda"))
    inside = cols < used[:, None]
    old = torch.where(inside, s["table"], 0).long().flatten()
    ref.scatter_add_(0, old, torch.where(inside, (children - 1)[:, None], 0).flatten())
    table = torch.where(cols < used[src][:, None], s["table"][src], -1)
    # reserve: one page for a sequence whose next token opens one, a copy for one whose last
    # page is shared (but for the last of the sharers, where nobody else holds it)
    part = lens % page != 0
    at = (lens // page).long()
    last = torch.where(part, torch.gather(table, 1, at[:, None])[:, 0], P).long()
    sharers = torch.zeros(P + 1, dtype=torch.int32, device="cuda").scatter_add_(
        0, last, torch.ones(S, dtype=torch.int32, device="cuda"))
    me = torch.arange(S, device="cuda")
    top = torch.full((P + 1,), -1, dtype=torch.int64, device="cuda").scatter_reduce_(0, last, me, "amax")
    held = torch.cat([ref, torch.zeros(1, dtype=torch.int32, device="cuda")])
    keeps = (sharers[last] == held[last]) & (top[last] == me)
    copies = part & ~keeps
    needs = copies | ~part
    rank = torch.cumsum(needs, 0) - 1
    free = torch.cumsum(ref == 0, 0)
    page_of = torch.searchsorted(free, rank + 1)
    new = torch.where(needs, page_of, last)
    table.scatter_(1, at[:, None], new.int()[:, None])
    ref.scatter_add_(0, torch.where(copies, last, 0), -copies.int())
    ref.scatter_add_(0, torch.where(needs, new, 0), needs.int())
    pool = s["pool"]
    to = torch.where(copies, new, torch.where(part, last, new))
    fr = torch.where(copies, last, to)
    pool[:, to] = pool[:, fr]
    # write: the new token's rows
    off = (lens % page).long()
    pool[0][new, off] = s["k_new"]
    pool[1][new, off] = s["v_new"]
    return {"table": table, "lens": lens, "ref": ref, "pool": pool}


def _run_plain_compact(s):
    c = s["case"]
    P, page = c["pages"], c["page"]
    ref, pool = s["ref"], s["pool"]
    live = ref > 0
    n_live = live.sum()
    ids = torch.arange(P, device="cuda")
    holes = torch.nonzero(~live & (ids < n_live))[:, 0]
    movers = torch.nonzero(live & (ids >= n_live))[:, 0]
    to = ids.clone()
    to[movers] = holes
    pool[:, holes] = pool[:, movers]
    used = (s["lens"] + page - 1) // page
    inside = torch.arange(s["table"].shape[1], device="cuda") < used[:, None]
    table = torch.where(inside, to[s["table"].long().clamp(min=0)].int(), -1)
    ref_out = torch.where(ids < n_live, ref, 0)
    ref_out[holes] = ref[movers]
    return {"table": table, "ref": ref_out, "n_live": n_live.int().view(1), "pool": pool}


# ---- the definitions in 64 bits -------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return globals()["_exact_" + case["op"]](case, s)


def _exact_select(case, s):
    B, K, V, N = case["batch"], case["beams"], case["vocab"], case["n_out"]
    out = {"parent": [], "token": [], "score": [], "finished": []}
    fin = s["finished"].cpu().numpy()
    lens = None if s["lengths"] is None else s["lengths"].cpu().numpy()
    for b in range(B):
        score = torch.full((K, V), -math.inf, dtype=torch.float64, device="cuda")
        rank = score.clone()
        for k in range(K):
            start = s["scores"][b, k].double()
            n = (0 if lens is None else int(lens[b, k])) + (0 if fin[b, k] else 1)
            if fin[b, k]:
                score[k, s["end"]] = start
            else:
                x = s["logits"][b * K + k].double() / case["temperature"]
                if s["allow"] is not None:
                    w = s["allow"][0 if s["allow"].shape[0] == 1 else b * K + k]
                    t = torch.arange(V, device="cuda")
                    x[((w[t // 32] >> (t % 32).int()) & 1) == 0] = -math.inf
                if bool((x > -math.inf).any()):
                    score[k] = torch.log_softmax(x, 0) + start
            rank[k] = score[k] / float(max(1, n)) ** case["alpha"]
        r, at = torch.sort(rank.flatten(), descending=True, stable=True)
        r, at = r[:N], at[:N]
        if at.numel() < N:
            r = torch.cat([r, r.new_full((N - at.numel(),), -math.inf)])
            at = torch.cat([at, at.new_zeros(N - at.numel())])
        ok = r > -math.inf
        par, tok = at // V, at % V
        done = (s["finished"][b].bool()[par] | (tok == s["end"])) & ok
        out["parent"].append(torch.where(ok, par, -1).int())
        out["token"].append(torch.where(ok, tok, -1))
        out["score"].append(torch.where(ok, score.flatten()[at], -math.inf))
        out["finished"].append(done.to(torch.uint8))
    return {k: torch.stack(v) for k, v in out.items()}


def _exact_attend(case, s):
    S, hq, hd = s["q"].shape
    group = hq // case["hkv"]
    out = torch.zeros((S, hq, hd), dtype=torch.float64, device="cuda")
    lse = torch.full((S, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n <= lo:
            continue
        t = torch.arange(lo, n, device="cuda")
        pages, rows = s["table"][i].long()[t // case["page"]], t % case["page"]
        k, v = s["k"][pages, rows].double(), s["v"][pages, rows].double()
        for h in range(case["hkv"]):
            x = s["q"][i, h * group:(h + 1) * group].double() @ k[:, h].T * s["scale"]
            lse[i, h * group:(h + 1) * group] = torch.logsumexp(x, 1)
            out[i, h * group:(h + 1) * group] = torch.softmax(x, 1) @ v[:, h]
    return {"out": out, "lse": lse}


def _exact_step(case, s):
    """By hand, sequence by sequence; the pool's pages are copied and not computed."""
    K, page, P = case["beams"], case["page"], case["pages"]
    old, ref = s["table"].cpu().numpy(), s["ref0"].cpu().numpy().copy()
    parent, n = s["parent"].cpu().numpy(), case["len"]
    used = -(-n // page)
    rows = [list(old[g * K + p, :used]) for g in range(case["groups"]) for p in parent[g]]
    for r in old:
        np.subtract.at(ref, r[:used], 1)
    for r in rows:
        np.add.at(ref, r, 1)
    free = [int(p) for p in np.flatnonzero(ref == 0)]
    moves = []
    if n % page:
        holders = {}
        for i, r in enumerate(rows):
            holders.setdefault(r[-1], []).append(i)
        for p, who in holders.items():
            if ref[p] == len(who):
                who.pop()
        copying = sorted(i for who in holders.values() for i in who)
        for i in copying:
            moves.append((rows[i][-1], free[0]))
            ref[rows[i][-1]] -= 1
            rows[i][-1] = free.pop(0)
            ref[rows[i][-1]] = 1
    else:
        for r in rows:
            r.append(free.pop(0))
            ref[r[-1]] = 1
    table = np.full(old.shape, -1, np.int32)
    for i, r in enumerate(rows):
        table[i, :len(r)] = r
    for a, b in moves:
        s["pool"][:, b] = s["pool"][:, a]
    for i, r in enumerate(rows):
        s["pool"][0, int(r[n // page]), n % page] = s["k_new"][i]
        s["pool"][1, int(r[n // page]), n % page] = s["v_new"][i]
    return {"table": torch.from_numpy(table), "lens": s["lens"], "ref": torch.from_numpy(ref), "pool": s["pool"]}


def _exact_compact(case, s):
    ref, table = s["ref"].cpu().numpy(), s["table"].cpu().numpy()
    used = -(-s["lens"].cpu().numpy() // case["page"])
    n_live = int((ref > 0).sum())
    holes = [p for p in range(n_live) if ref[p] == 0]
    movers = [p for p in range(n_live, case["pages"]) if ref[p] > 0]
    to = {p: p for p in range(case["pages"])}
    new_ref = ref.copy()
    new_ref[n_live:] = 0
    for h, m in zip(holes, movers):
        to[m] = h
        new_ref[h] = ref[m]
        s["pool"][:, h] = s["pool"][:, m]
    out = np.full(table.shape, -1, np.int32)
    for i in range(table.shape[0]):
        out[i, :used[i]] = [to[int(p)] for p in table[i, :used[i]]]
    return {"table": torch.from_numpy(out), "ref": torch.from_numpy(new_ref),
            "n_live": torch.tensor([n_live], dtype=torch.int32), "pool": s["pool"]}


if __name__ == "__main__":
    for one in listed() + [draw(random.Random(i)) for i in range(20)]:
        print(one.get("name", one), work(one))
