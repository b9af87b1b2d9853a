"""The losses of sampled and compared sequences in 64 bits: a plain reference, written from their definitions.

Inputs are torch tensors on any device; everything is computed in double on that device.  ``policy`` and ``preference``
return the outputs of the calls of the same name, ``slope``, d total / d logp per row, from autograd, and ``mass``, the sum of the
magnitudes of the terms that make up the slope (what its rounding is relative to where they cancel)."""
import torch


def logprobs(x, targets, on):
    """logp of counted rows (0 elsewhere) of scaled logits x in double."""
    lp = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    rows = torch.nonzero(on)[:, 0]
    if len(rows):
        lse = torch.logsumexp(x[rows], -1)
        hit = x[rows, targets[rows]]
        lp[rows] = torch.where(hit == -torch.inf, hit, hit - lse)
    return lp


def counted(n, first, mask, device):
    on = torch.ones(n, dtype=torch.bool, device=device) if mask is None else mask.to(device) != 0
    if first is not None:
        row = torch.arange(n, device=device)
        on = on & (row >= int(first[0])) & (row < int(first[-1]))
    return on


def groups(n, first, on):
    if first is None:
        return [torch.nonzero(on)[:, 0]]
    f = first.tolist()
    return [torch.nonzero(on[a:b])[:, 0] + a for a, b in zip(f[:-1], f[1:])]


def policy(lp, on, first, adv, old, ref, low=0.2, high=0.2, kl=0.0, seq_ratio=False, seq_mean=False, seq_adv=False,
           summed=False):
    n = lp.shape[0]
    x = lp.detach().clone().requires_grad_()
    gs = groups(n, first, on)
    some, total_n = sum(1 for g in gs if len(g)), int(on.sum())
    zero = torch.zeros((), dtype=torch.float64, device=lp.device)
    per_token = torch.zeros(n, dtype=torch.float64, device=lp.device)
    mass = torch.zeros(n, dtype=torch.float64, device=lp.device)
    sums = [zero, zero, zero]
    for s, g in enumerate(gs):
        if not len(g):
            continue
        if seq_mean:
            w = 1.0 / len(g) if summed else 1.0 / (len(g) * some)
        else:
            w = 1.0 if summed else 1.0 / total_n
        delta = x[g] - (old[g].double() if old is not None else x[g].detach())
        if seq_ratio:
            delta = delta.mean().expand(len(g))
        a = adv[s].double().expand(len(g)) if seq_adv else adv[g].double()
        r = torch.exp(delta)
        edge = torch.where(a > 0, 1.0 + high, 1.0 - low)
        out = torch.where(a > 0, r > edge, r < edge) & (a != 0)
        term = torch.where(a == 0, zero, -a * torch.where(out, edge, r))
        sums[0] = sums[0] + w * term.sum()
        sums[2] = sums[2] + w * out.double().sum()
        part = (a * r).abs().detach() * (~out & (a != 0))
        mass[g] = w * (part.mean() if seq_ratio else part)
        if ref is not None:
            q = ref[g].double() - x[g]
            k = torch.expm1(q) - q
            sums[1] = sums[1] + w * k.sum()
            if kl > 0:
                term = term + kl * k
                mass[g] += w * kl * (torch.exp(q.detach()) + 1.0)
        per_token[g] = term.detach()
    total = sums[0] + kl * sums[1] if kl > 0 else sums[0]
    if total.requires_grad:
        total.backward()
    slope = x.grad if x.grad is not None else torch.zeros_like(lp)
    return {"scalars": torch.stack([total, *sums]).detach(), "per_token": per_token, "logp": torch.where(on, lp, 0.0),
            "slope": slope, "mass": mass}


def preference(lp, on, first, ref, objective="sigmoid", beta=0.1, margin=0.0, smoothing=0.0, nll=0.0, length_mean=False,
               summed=False):
    n = lp.shape[0]
    x = lp.detach().clone().requires_grad_()
    gs = groups(n, first, on)
    half = len(gs) // 2
    zero = torch.zeros((), dtype=torch.float64, device=lp.device)
    value = []
    for g in gs:
        v = (x[g] - (ref[g].double() if ref is not None else 0.0)).sum()
        value.append(v / max(1, len(g)) if length_mean else v)
    live = [i for i in range(half) if len(gs[i]) and len(gs[half + i])]
    per_pair, mean, right = torch.zeros(half, dtype=torch.float64, device=lp.device), zero, 0.0
    mass = torch.zeros(n, dtype=torch.float64, device=lp.device)
    for i in live:
        u = value[i] - value[half + i]
        if objective == "squared":
            term = (u - 0.5 / beta) ** 2
        elif objective == "hinge":
            term = torch.clamp(1.0 - beta * u, min=0.0)
        else:
            h = beta * u - margin
            term = (1.0 - smoothing) * torch.nn.functional.softplus(-h, threshold=1e4)
            if smoothing > 0:
                term = term + smoothing * torch.nn.functional.softplus(h, threshold=1e4)
        per_pair[i] = term.detach()
        if objective == "squared":
            size = 2.0 * (u.detach().abs() + 0.5 / beta)
        elif objective == "hinge":
            size = beta if float(beta * u.detach()) < 1.0 else 0.0
        else:
            size = beta * ((1.0 - smoothing) * torch.sigmoid(-h.detach()) + smoothing * torch.sigmoid(h.detach()))
        for s in (i, half + i):
            mass[gs[s]] += size / (1 if summed else len(live)) / (len(gs[s]) if length_mean else 1)
        mean, right = mean + term, right + float(u.detach() > 0)
    chosen = torch.cat([torch.zeros(0, dtype=torch.int64, device=lp.device), *gs[:half]])
    like = -x[chosen].sum()
    if not summed:
        mean, right = mean / max(1, len(live)), right / max(1, len(live))
        like = like / max(1, len(chosen))
    total = mean + nll * like if nll > 0 else mean
    mass[chosen] += nll / (1 if summed else max(1, len(chosen)))
    if total.requires_grad:
        total.backward()
    slope = x.grad if x.grad is not None else torch.zeros_like(lp)
    right = torch.tensor(right, dtype=torch.float64, device=lp.device)
    return {"scalars": torch.stack([total, mean, like, right]).detach(), "per_pair": per_pair,
            "log_ratio": torch.stack(value).detach(), "logp": torch.where(on, lp, 0.0), "slope": slope,
            "mass": mass}


def grad_logits(x, targets, on, slope, temperature=1.0):
    """d total / d logits of scaled logits x, rows that do not count zero; and the coefficient a per row."""
    a = torch.where(on, -slope / temperature, 0.0)
    g = torch.zeros_like(x)
    rows = torch.nonzero(on & (a != 0))[:, 0]
    if len(rows):
        p = torch.softmax(x[rows], -1)
        p[torch.arange(len(rows), device=x.device), targets[rows]] -= 1.0
        g[rows] = a[rows, None] * torch.where(torch.isnan(p), 0.0, p)
    return g, a
