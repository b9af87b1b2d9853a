"""The losses on log-probabilities of whole sequences, each as one measured pass, forward and backward.

Two losses, each in two forms:

  policy      the clipped policy loss with a KL term against a reference model, over
              sampled tokens (lossk_policy_fwd_bwd from hidden rows and the head's
              weight, lossk_policy_from_logits from given logits)
  preference  paired log ratios of chosen and rejected sequences
              (lossk_preference_fwd_bwd, lossk_preference_from_logits)

With ``own`` false a pass runs the loss's plain form in elementary torch
operations; with ``own`` true it calls the package.  ``exact`` is the
definition in 64 bits, written apart from the plain form.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---- the cases -----------------------------------------------------------------

def _policy(name, n, d, vocab, dtype, **more):
    case = {"name": name, "op": "policy", "n": n, "d": d, "vocab": vocab, "dtype": dtype, "seqs": 0, "prompt": 0.0,
            "tail": 0, "ratio": "token", "mean": "token", "low": 0.2, "high": 0.2, "kl": 0.04, "temperature": 1.0}
    return {**case, **more}


def _preference(name, n, d, vocab, dtype, pairs, **more):
    case = {"name": name, "op": "preference", "n": n, "d": d, "vocab": vocab, "dtype": dtype, "seqs": 2 * pairs,
            "prompt": 0.0, "tail": 0, "objective": "sigmoid", "beta": 0.1, "margin": 0.0, "smoothing": 0.0, "nll": 0.0,
            "length_mean": False}
    return {**case, **more}


def listed():
    return [
        # A micro-batch of short answers over a mid-sized vocabulary: all latency.
        _policy("policy logits 48 x 32000, bf16", 48, 0, 32000, "bf16", seqs=6),
        # Eight sampled answers and their prompts, whose rows do not count, at a large vocabulary.
        _policy("policy logits 2048 x 151936, bf16", 2048, 0, 151936, "bf16", seqs=8, prompt=0.2, high=0.28),
        # Ratios of whole sequences in fp32 with an odd vocabulary, a sampling temperature, rows of padding behind
        # the last sequence.
        _policy("policy logits 1531 x 32003, f32, sequences", 1531, 0, 32003, "f32", seqs=11, prompt=0.1, tail=40,
                ratio="sequence", mean="sequence", low=3e-3, high=4e-3, temperature=0.7),
        # Three short pairs, rows that are not 16-byte aligned, label smoothing.
        _preference("preference logits 300 x 32003, f16", 300, 0, 32003, "f16", 3, prompt=0.3, smoothing=0.1),
        # Sixteen pairs of full answers with their prompts, and the likelihood of the chosen ones beside them.
        _preference("preference logits 4096 x 151936, bf16", 4096, 0, 151936, "bf16", 16, prompt=0.3, nll=0.2),
        # A tiny model in fp32: tokens without sequences, advantages token by token.
        _policy("policy head 64 x 64 x 1000, f32", 64, 64, 1000, "f32", kl=0.0),
        # A small head, one micro-batch.
        _policy("policy head 512 x 1024 x 32000, bf16", 512, 1024, 32000, "bf16", seqs=4, temperature=0.9),
        # A 0.6B model's head: eight answers of up to 256 tokens, every row counts.
        _policy("policy head 2048 x 1024 x 151936, bf16", 2048, 1024, 151936, "bf16", seqs=8, ratio="sequence",
                mean="sequence", low=3e-3, high=4e-3),
        # The widest head: a batch of long answers behind prompts of a quarter of the rows.
        _policy("policy head 8192 x 4096 x 128256, bf16", 8192, 4096, 128256, "bf16", seqs=16, prompt=0.25),
        # Two ragged pairs and a small head in fp16, averaged log ratios against a squared target.
        _preference("preference head 203 x 264 x 5000, f16", 203, 264, 5000, "f16", 2, prompt=0.2, objective="squared",
                    length_mean=True),
        # Four pairs on a small head, hinge loss, no prompt.
        _preference("preference head 1000 x 1024 x 32000, f16", 1000, 1024, 32000, "f16", 4, objective="hinge", beta=0.05),
        # Sixteen pairs, half of their rows prompts, on a 2048-wide head.
        _preference("preference head 4096 x 2048 x 151936, bf16", 4096, 2048, 151936, "bf16", 16, prompt=0.5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["policy", "preference"])
    head = rng.random() < 0.5
    # fp32 heads are small: the matrix products of large ones run in 16 bits
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    n, vocab, d = _log_int(rng, 16, 8192), _log_int(rng, 500, 151936), 0
    if head:
        d = 8 * _log_int(rng, 8, 512)
        if dtype == "f32":
            n, vocab, d = min(n, 128), min(vocab, 4000), min(d, 256)
        while n * d * vocab > 2.0e12:
            n //= 2
    while n * vocab * ESIZE[dtype] > 1.24e9:
        n //= 2
    n = max(n, 8)
    tail = rng.choice([0, 0, rng.randint(0, n // 8)])
    prompt = rng.choice([0.0, rng.uniform(0.0, 0.6)])
    if op == "policy":
        seqs = rng.choice([0, _log_int(rng, 1, max(1, n // 8))])
        ratio = rng.choice(["token", "sequence"]) if seqs else "token"
        narrow = ratio == "sequence"
        case = _policy("", n, d, vocab, dtype, seqs=seqs, tail=tail if seqs else 0, prompt=prompt, ratio=ratio,
                       mean=rng.choice(["token", "sequence"]) if seqs else "token",
                       low=rng.uniform(2e-3, 1e-2) if narrow else rng.uniform(0.1, 0.3),
                       high=rng.uniform(2e-3, 1e-2) if narrow else rng.uniform(0.1, 0.4),
                       kl=rng.choice([0.0, rng.uniform(0.001, 0.2)]),
                       temperature=rng.choice([1.0, rng.uniform(0.5, 1.5)]))
    else:
        objective = rng.choice(["sigmoid", "sigmoid", "hinge", "squared"])
        case = _preference("", n, d, vocab, dtype, _log_int(rng, 1, max(1, n // 16)), tail=tail, prompt=prompt,
                           objective=objective, beta=rng.uniform(0.03, 0.5),
                           margin=rng.choice([0.0, rng.uniform(0.0, 1.0)]) if objective == "sigmoid" else 0.0,
                           smoothing=rng.choice([0.0, rng.uniform(0.0, 0.3)]) if objective == "sigmoid" else 0.0,
                           nll=rng.choice([0.0, rng.uniform(0.05, 1.0)]), length_mean=rng.choice([False, True]))
    del case["name"]
    return case


# ---- what the cases share ---------------------------------------------------------

def _layout(case):
    """(first row of each sequence and the end, rows that count), of the case's sizes alone."""
    n, seqs = case["n"], case["seqs"]
    r = np.random.default_rng([n, seqs, case["vocab"]])
    counts = np.ones(n, dtype=np.uint8)
    if not seqs:
        counts[r.random(n) < case["prompt"]] = 0
        return None, counts
    rows = n - case["tail"]
    # ragged: shares of the rows between one half and three halves of the mean
    ends = np.cumsum(r.uniform(0.5, 1.5, seqs))
    first = np.concatenate([[0], np.floor(ends / ends[-1] * rows + 0.5)]).astype(np.int32)
    for a, b in zip(first[:-1], first[1:]):
        counts[a:a + int((b - a) * case["prompt"])] = 0
    return first, counts


def work(case):
    n, d, vocab, es = case["n"], case["d"], case["vocab"], ESIZE[case["dtype"]]
    first, counts = _layout(case)
    live = int((counts[:first[-1]] if first is not None else counts).sum())
    per_row = 8 + 1 + 2 * 4 + 2 * 4
    if d:
        # what is read: the rows that count and the weight; written: both gradients
        return {"bytes": (live * d + vocab * d) * es + (n * d + vocab * d) * es + n * per_row, "flops": 6 * live * d * vocab}
    return {"bytes": (live + n) * vocab * es + n * per_row, "flops": 8 * live * vocab}


def _rows(count, vocab):
    """Blocks of rows whose fp32 logits take at most a quarter of a GB."""
    step = max(1, (1 << 26) // vocab)
    return [(i, min(i + step, count)) for i in range(0, count, step)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng([seed, 29])
    n, d, vocab, dtype = case["n"], case["d"], case["vocab"], DTYPES[case["dtype"]]
    T = case.get("temperature", 1.0)
    s = {"case": case}
    # logits of standard deviation 2.5, so that a sampled token's probability is neither near 0 nor near 1
    if d:
        s["hidden"] = torch.randn((n, d), device="cuda", generator=gen).to(dtype)
        s["weight"] = (torch.randn((vocab, d), device="cuda", generator=gen) * (2.5 / math.sqrt(d))).to(dtype)
        wide = s["weight"].float()
    else:
        s["logits"] = torch.empty((n, vocab), device="cuda", dtype=dtype)
    target = torch.empty(n, dtype=torch.int64, device="cuda")
    logp = torch.empty(n, dtype=torch.float64, device="cuda")
    for a, b in _rows(n, vocab):
        if d:
            x = s["hidden"][a:b].float() @ wide.t()
        else:
            s["logits"][a:b] = torch.randn((b - a, vocab), device="cuda", generator=gen) * 2.5
            x = s["logits"][a:b].float()
        # the tokens are the model's own samples
        target[a:b] = torch.multinomial(torch.softmax(x / T, -1), 1, generator=gen)[:, 0]
        if d:
            logp[a:b] = torch.log_softmax(x / T, -1).gather(1, target[a:b, None])[:, 0]
        else:
            logp[a:b] = torch.log_softmax(x.double() / T, -1).gather(1, target[a:b, None])[:, 0]
    first, counts = _layout(case)
    s["mask"] = torch.from_numpy(counts).cuda()
    s["first"] = torch.from_numpy(first).cuda() if first is not None else None
    logp = logp.cpu().numpy()
    spans = list(zip(first[:-1], first[1:])) if first is not None else []
    if case["op"] == "policy":
        # the sampling policy is a few updates old, the reference model further away
        narrow = case["ratio"] == "sequence"
        delta = rng.normal(0.0, 0.15, n)
        if narrow:
            for a, b in spans:
                on = counts[a:b] == 1
                if on.any():
                    delta[a:b] += rng.normal(0.0, case["high"]) - delta[a:b][on].mean()
        lo, hi = math.log(1.0 - case["low"]), math.log(1.0 + case["high"])
        near = 2e-4 if not narrow else 2e-5
        # a ratio that rounding could put on either side of a border is moved off it
        for border in (lo, hi):
            if narrow:
                for a, b in spans:
                    on = counts[a:b] == 1
                    if on.any() and abs(delta[a:b][on].mean() - border) < near:
                        delta[a:b] += 2 * near
            else:
                delta[np.abs(delta - border) < near] += 2 * near
        s["old"] = torch.from_numpy((logp - delta).astype(np.float32)).cuda()
        s["ref"] = torch.from_numpy((logp + rng.normal(0.0, 0.4, n)).astype(np.float32)).cuda()
        s["advantages"] = torch.from_numpy(rng.normal(0.0, 1.0, len(spans) if spans else n).astype(np.float32)).cuda()
    else:
        ref = logp + rng.normal(0.0, 0.3, n)
        for a, b in spans:
            ref[a:b] += rng.normal(0.0, 0.1)
        diffs = [((logp - ref)[a:b])[counts[a:b] == 1] for a, b in spans]
        value = [(x.mean() if case["length_mean"] else x.sum()) if len(x) else 0.0 for x in diffs]
        half = len(spans) // 2
        for i in range(half):
            u = value[i] - value[half + i]
            # a pair that rounding could put on either side of a tie or of the hinge is moved off it
            for border in (0.0, 1.0 / case["beta"]):
                if abs(u - border) < 2e-3 and len(diffs[i]):
                    a, b = spans[i]
                    ref[a:b] -= 5e-3 / (1 if case["length_mean"] else len(diffs[i]))
        s["ref"] = torch.from_numpy(ref.astype(np.float32)).cuda()
    # rows that do not count carry no label
    target[s["mask"] == 0] = -100
    if first is not None:
        target[int(first[-1]):] = -100
    s["targets"] = target
    if own:
        _own_state(case, s)
    return s


# ---- the package's calls, on buffers and a workspace that a training loop keeps ------

def _own_state(case, s):
    import output_projection_cross_gb300 as L
    code = {"f32": L.F32, "bf16": L.BF16, "f16": L.F16}[case["dtype"]]
    n, d, vocab, seqs = case["n"], case["d"], case["vocab"], case["seqs"]
    kind = L.KIND_SEQUENCE_HEAD if d else L.KIND_SEQUENCE_LOGITS
    s["L"] = L
    s["out"] = {"ws": L.sequence_workspace(kind, n, d if d else 1, vocab, seqs, code)}
    if d:
        s["out"]["d_hidden"] = torch.empty_like(s["hidden"])
        s["out"]["d_weight"] = torch.empty_like(s["weight"])
    else:
        s["out"]["grad_logits"] = torch.empty_like(s["logits"])
    for name, size in (("scalars_out", 4), ("logp_out", n),
                       *((("per_token_out", n),) if case["op"] == "policy" else
                         (("per_pair_out", seqs // 2), ("log_ratio_out", seqs)))):
        s["out"][name] = torch.empty(size, dtype=torch.float32, device="cuda")


def _run_own(s):
    c, L = s["case"], s["L"]
    given = (s["hidden"], s["weight"]) if c["d"] else (s["logits"],)
    if c["op"] == "policy":
        flags = (L.SEQ_ADVANTAGES if c["seqs"] else 0) | (L.SEQ_RATIO if c["ratio"] == "sequence" else 0) | (
            L.SEQ_MEAN if c["mean"] == "sequence" else 0)
        call = L.lossk_policy_fwd_bwd if c["d"] else L.lossk_policy_from_logits
        r = call(*given, s["targets"], s["advantages"], old_logp=s["old"], ref_logp=s["ref"] if c["kl"] else None,
                 first=s["first"], loss_mask=s["mask"], clip_low=c["low"], clip_high=c["high"], kl_weight=c["kl"],
                 temperature=c["temperature"], flags=flags, **s["out"])
        keys = ["scalars", "per_token", "logp"]
    else:
        call = L.lossk_preference_fwd_bwd if c["d"] else L.lossk_preference_from_logits
        r = call(*given, s["targets"], s["first"], ref_logp=s["ref"], loss_mask=s["mask"], objective=c["objective"],
                 beta=c["beta"], margin=c["margin"], label_smoothing=c["smoothing"], nll_weight=c["nll"],
                 flags=L.LENGTH_MEAN if c["length_mean"] else 0, **s["out"])
        keys = ["scalars", "per_pair", "log_ratio", "logp"]
    return {k: r[k] for k in keys + (["d_hidden", "d_weight"] if c["d"] else ["grad_logits"])}


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---- the plain forms -----------------------------------------------------------------

def _seq_sums(s, v):
    """Sums over each sequence's rows, in 64 bits, and each row's sequence."""
    total = torch.cat([torch.zeros(1, dtype=torch.float64, device="cuda"), v.double().cumsum(0)])
    first = s["first"].long()
    return total[first[1:]] - total[first[:-1]]


def _seq_of(s, n):
    """Each row's sequence (the last one's for rows behind it)."""
    row = torch.arange(n, device="cuda")
    return (torch.searchsorted(s["first"].long(), row, right=True) - 1).clamp(0, s["case"]["seqs"] - 1)


def _plain_policy(s, logp, on):
    c, n = s["case"], logp.shape[0]
    delta = torch.where(on, logp - s["old"], torch.zeros_like(logp))
    one = on.double()
    seq = _seq_of(s, n) if c["seqs"] else None
    count = _seq_sums(s, one).clamp(min=1) if c["seqs"] else None
    if c["ratio"] == "sequence":
        delta = (_seq_sums(s, delta) / count)[seq].float()
    adv = s["advantages"][seq] if c["seqs"] else s["advantages"]
    if c["mean"] == "sequence":
        with_any = (_seq_sums(s, one) > 0).sum().clamp(min=1)
        w = torch.where(on, (1.0 / (with_any * count))[seq], torch.zeros_like(one))
    else:
        w = one / one.sum().clamp(min=1)
    ratio = torch.exp(delta)
    free, held = ratio * adv, ratio.clamp(1.0 - c["low"], 1.0 + c["high"]) * adv
    loss = -torch.minimum(free, held)
    clipped = free > held
    slope = torch.where(clipped, torch.zeros_like(free), -free).double() * w
    if c["ratio"] == "sequence":
        slope = torch.where(on, (_seq_sums(s, slope) / count)[seq], torch.zeros_like(slope))
    policy = (loss * w).sum()
    kl_mean = torch.zeros_like(policy)
    if c["kl"]:
        gap = torch.where(on, s["ref"] - logp, torch.zeros_like(logp))
        kl = torch.exp(gap) - gap - 1.0
        kl_mean = (kl * w).sum()
        loss = loss + c["kl"] * kl
        slope = slope + c["kl"] * (1.0 - torch.exp(gap)) * w
    scalars = torch.stack([policy + c["kl"] * kl_mean, policy, kl_mean, (clipped * w).sum()]).float()
    return slope.float(), {"scalars": scalars, "per_token": torch.where(on, loss, torch.zeros_like(loss)),
                           "logp": torch.where(on, logp, torch.zeros_like(logp))}


def _plain_preference(s, logp, on):
    c, n = s["case"], logp.shape[0]
    half = c["seqs"] // 2
    one = on.double()
    seq, count = _seq_of(s, n), _seq_sums(s, one)
    ratio = _seq_sums(s, torch.where(on, (logp - s["ref"]).double(), torch.zeros_like(one)))
    per = 1.0 / count.clamp(min=1) if c["length_mean"] else torch.ones_like(count)
    ratio = ratio * per
    live = ((count[:half] > 0) & (count[half:] > 0)).double()
    u = ratio[:half] - ratio[half:]
    if c["objective"] == "squared":
        loss, slope = (u - 0.5 / c["beta"]) ** 2, 2.0 * (u - 0.5 / c["beta"])
    elif c["objective"] == "hinge":
        h = c["beta"] * u
        loss, slope = (1.0 - h).clamp(min=0), torch.where(h < 1.0, -c["beta"], 0.0).double()
    else:
        h, e = c["beta"] * u - c["margin"], c["smoothing"]
        soft = lambda x: x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))  # noqa: E731
        loss = (1.0 - e) * soft(-h) + e * soft(h)
        slope = c["beta"] * (1.0 / (1.0 + torch.exp(-h)) - (1.0 - e))
    pairs = live.sum().clamp(min=1)
    slope = torch.cat([slope * live, -slope * live]) * per / pairs
    mean = (loss * live).sum() / pairs
    chosen = on & (seq < half)
    chosen_n = chosen.sum().clamp(min=1)
    nll = torch.where(chosen, -logp, torch.zeros_like(logp)).sum(dtype=torch.float64) / chosen_n
    by_row = torch.where(on, slope[seq], torch.zeros_like(one)) - c["nll"] * chosen.double() / chosen_n
    scalars = torch.stack([mean + c["nll"] * nll, mean, nll, ((u > 0) * live).sum() / pairs]).float()
    return by_row.float(), {"scalars": scalars, "per_pair": (loss * live).float(), "log_ratio": ratio.float(),
                            "logp": torch.where(on, logp, torch.zeros_like(logp))}


def _run_plain(s):
    c = s["case"]
    T = c.get("temperature", 1.0)
    n = c["n"]
    row = torch.arange(n, device="cuda")
    on = s["mask"] != 0
    if c["seqs"]:
        on = on & (row < s["first"][-1])
    y = s["targets"].clamp(min=0)
    # a token's own logit in 64 bits: sequences' sums of log ratios cancel
    if c["d"]:
        h, w = s["hidden"].float(), s["weight"].float()
        x = (h @ w.t()) / T
        hit = (h.double() * w[y].double()).sum(-1) / T
    else:
        x = s["logits"].float() / T
        hit = s["logits"][row, y].double() / T
    m = x.amax(-1, keepdim=True)
    x -= m
    p = x.exp_()
    z = p.sum(-1)
    logp = (hit - m[:, 0].double() - torch.log(z.double())).float()
    slope, out = (_plain_policy if c["op"] == "policy" else _plain_preference)(s, logp, on)
    # d loss / d logits = slope (one-hot - softmax) / T
    a = slope / T
    p *= (-a / z)[:, None]
    p[row, y] += a
    dtype = DTYPES[c["dtype"]]
    if c["d"]:
        out["d_hidden"] = (p @ w).to(dtype)
        out["d_weight"] = (p.t() @ h).to(dtype)
    else:
        out["grad_logits"] = p.to(dtype)
    return out


# ---- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    global own
    n, d, vocab = case["n"], case["d"], case["vocab"]
    if d and n * d * vocab > 1.4e12:
        return None
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    T = case.get("temperature", 1.0)
    first, counts = _layout(case)
    live = torch.from_numpy(np.flatnonzero(counts[:int(first[-1])] if first is not None else counts)).cuda()
    y = s["targets"][live]
    if d:
        weight = s["weight"].double()
        rows = lambda i: s["hidden"][live[i]].double() @ weight.t() / T  # noqa: E731
    else:
        rows = lambda i: s["logits"][live[i]].double() / T  # noqa: E731
    blocks = [slice(a, b) for a, b in _rows(len(live), vocab)]
    logp = torch.zeros(n, dtype=torch.float64, device="cuda")
    for i in blocks:
        logp[live[i]] = torch.log_softmax(rows(i), -1).gather(1, y[i, None])[:, 0]
    # the loss of the log-probabilities, sequence by sequence on the host, and its derivative
    lp = logp.cpu().requires_grad_()
    out = (_exact_policy if case["op"] == "policy" else _exact_preference)(case, s, lp, live.cpu(), first)
    out["scalars"][0].backward()
    slope = lp.grad.cuda()[live] / T
    out = {k: v.detach() for k, v in out.items()}
    out["logp"] = logp.cpu()
    if d:
        dh = torch.zeros((n, d), dtype=torch.float64, device="cuda")
        dw = torch.zeros((vocab, d), dtype=torch.float64, device="cuda")
    else:
        dl = torch.zeros((n, vocab), dtype=torch.float64, device="cuda")
    for i in blocks:
        g = torch.softmax(rows(i), -1) * -slope[i, None]
        g[torch.arange(g.shape[0], device="cuda"), y[i]] += slope[i]
        if d:
            dh[live[i]] = g @ weight
            dw += g.t() @ s["hidden"][live[i]].double()
        else:
            dl[live[i]] = g
    if d:
        out["d_hidden"], out["d_weight"] = dh, dw
    else:
        out["grad_logits"] = dl
    return out


def _exact_policy(case, s, lp, live, first):
    n = case["n"]
    old, ref, adv = s["old"].cpu().double(), s["ref"].cpu().double(), s["advantages"].cpu().double()
    mine = torch.zeros(n, dtype=torch.bool)
    mine[live] = True
    if first is None:
        groups = [torch.nonzero(mine)[:, 0]]
        advs = [adv[groups[0]]]
    else:
        groups = [torch.nonzero(mine[int(a):int(b)])[:, 0] + int(a) for a, b in zip(first[:-1], first[1:])]
        advs = [adv[i].expand(len(g)) for i, g in enumerate(groups)]
    some = sum(1 for g in groups if len(g))
    per_token = torch.zeros(n, dtype=torch.float64)
    policy, kl_mean, clip = [torch.zeros((), dtype=torch.float64) for _ in range(3)]
    for g, a in zip(groups, advs):
        if not len(g):
            continue
        w = 1.0 / (some * len(g)) if case["mean"] == "sequence" else 1.0 / len(live)
        delta = lp[g] - old[g]
        if case["ratio"] == "sequence":
            delta = delta.mean().expand(len(g))
        r = delta.exp()
        inside = torch.where(a >= 0, r <= 1.0 + case["high"], r >= 1.0 - case["low"])
        border = torch.where(a >= 0, 1.0 + case["high"], 1.0 - case["low"]).double()
        term = -a * torch.where(inside, r, border)
        policy = policy + w * term.sum()
        clip = clip + w * (~inside).double().sum()
        if case["kl"]:
            q = ref[g] - lp[g]
            kl = torch.expm1(q) - q
            kl_mean = kl_mean + w * kl.sum()
            term = term + case["kl"] * kl
        per_token[g] = term.detach()
    return {"scalars": torch.stack([policy + case["kl"] * kl_mean, policy, kl_mean, clip]), "per_token": per_token}


def _exact_preference(case, s, lp, live, first):
    ref = s["ref"].cpu().double()
    mine = torch.zeros(case["n"], dtype=torch.bool)
    mine[live] = True
    groups = [torch.nonzero(mine[int(a):int(b)])[:, 0] + int(a) for a, b in zip(first[:-1], first[1:])]
    half = len(groups) // 2
    value = [(lp[g] - ref[g]).sum() / (max(1, len(g)) if case["length_mean"] else 1) for g in groups]
    used = [i for i in range(half) if len(groups[i]) and len(groups[half + i])]
    zero = torch.zeros((), dtype=torch.float64)
    per_pair, mean, right = [zero] * half, zero, 0
    for i in used:
        u = value[i] - value[half + i]
        right += bool(u > 0)
        if case["objective"] == "squared":
            term = (u - 1.0 / (2.0 * case["beta"])).square()
        elif case["objective"] == "hinge":
            term = torch.relu(1.0 - case["beta"] * u)
        else:
            h = case["beta"] * u - case["margin"]
            term = -(1.0 - case["smoothing"]) * torch.nn.functional.logsigmoid(h) - case["smoothing"] * \
                torch.nn.functional.logsigmoid(-h)
        per_pair[i] = term
        mean = mean + term / len(used)
    chosen = torch.cat([zero.reshape(1)[:0].long(), *groups[:half]])
    nll = -lp[chosen].sum() / max(1, len(chosen))
    return {"scalars": torch.stack([mean + case["nll"] * nll, mean, nll,
                                    torch.tensor(right / max(1, len(used)), dtype=torch.float64)]),
            "per_pair": torch.stack(per_pair), "log_ratio": torch.stack(value)}
