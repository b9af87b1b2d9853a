"""The policy and preference losses on the GPU against their definitions in 64 bits (seq_ref), from given logits and
from hidden rows and the head's weight: types, sizes, masks, options.

Tolerances.  logp from given logits: the exponentials' arguments are one fp32 rounding of a value below 64 in log2 units
(2^-18 ln 2 < 3e-6), a thread's sum and the tree have below 64 additions (64 * 2^-24 < 4e-6), ex2.approx and log2f less
than 2^-21 together: 8e-6 and the output's own rounding.  From hidden rows the logits carry fp32 sums of d_model
products, d / 16 + 8 additions (each truncating, 2^-23) to partial sums of at most twice the largest logit.  A
coefficient is a sum of terms: it is as far off as logp times its derivative, at most 8 times the sum of their
magnitudes (seq_ref's mass; not its own size, which cancels where the policy's and the KL's terms meet).  In the
preference loss it moves with its pair's log ratio: d log |slope| / du is at most beta (sigmoid) and the slope 2 (u - 1 /
(2 beta)) is 2 far off u's error, 4 beta times its mass (squared).  A gradient element is rounded once to its type
(half a step), and in the 16-bit heads the grad tile's elements once more."""
import math

import pytest
import torch

import output_projection_cross_gb300 as L
import seq_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODE = {"bf16": L.BF16, "f16": L.F16, "f32": L.F32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def splits(n, k, seed, tail=0, empty=False):
    """first of k ragged sequences over n - tail rows (one of them empty)."""
    r = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(0, n - tail + 1, (k - 1,), generator=r)).values
    if empty and k > 2:
        cuts[1] = cuts[0]
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([n - tail])]).int().cuda()


class Case:
    def __init__(self, n, V, dtype, d=0, seqs=0, masked=0.0, tail=0, empty=False, T=1.0, std=2.5, seed=0):
        g = gen(seed)
        self.n, self.V, self.d, self.dtype, self.T = n, V, d, dtype, T
        if d:
            self.hidden = torch.randn(n, d, device="cuda", generator=g).to(DT[dtype])
            self.weight = (torch.randn(V, d, device="cuda", generator=g) * (std / math.sqrt(d))).to(DT[dtype])
            self.x = self.hidden.double() @ self.weight.double().t() / T
        else:
            self.logits = (torch.randn(n, V, device="cuda", generator=g) * std).to(DT[dtype])
            self.x = self.logits.double() / T
        self.targets = torch.randint(0, V, (n,), device="cuda", generator=g)
        self.first = splits(n, seqs, seed, tail, empty) if seqs else None
        self.mask = (torch.rand(n, device="cuda", generator=g) >= masked).to(torch.uint8) if masked else None
        self.fill(g)

    def fill(self, g):
        n = self.n
        self.on = R.counted(n, self.first.cpu() if self.first is not None else None, self.mask, "cuda")
        self.lp = R.logprobs(self.x, self.targets, self.on)
        noise = torch.randn(n, device="cuda", generator=g, dtype=torch.float64)
        # no ratio within 2e-3 of a border of the clamp at 0.2
        near = lambda b: (noise * 0.15 - math.log(b)).abs() < 2e-3  # noqa: E731
        noise = torch.where(near(0.8) | near(1.2), noise + 0.1, noise)
        self.old = (self.lp - 0.15 * noise).float()
        self.ref = (self.lp + 0.4 * torch.randn(n, device="cuda", generator=g, dtype=torch.float64)).float()
        self.adv = torch.randn(n, device="cuda", generator=g)
        off = ~self.on                       # what rows that do not count hold does not matter
        for t, bad in ((self.old, math.nan), (self.ref, math.inf), (self.adv, -math.inf)):
            t[off] = bad
        self.targets[off] = -100
        if not self.d:
            self.logits[off] = math.nan
        else:
            self.hidden[off] = math.nan

    def lp_tol(self):
        if not self.d:
            return 8e-6 / min(1.0, self.T)
        top = float(self.x[self.on].abs().max()) if self.on.any() else 0.0
        if self.dtype == "f32":
            return 8e-6 / min(1.0, self.T) + top * 2.0 ** -22
        return 8e-6 / min(1.0, self.T) + (self.d / 16 + 8) * 2.0 ** -23 * 2 * top


def close(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~torch.isclose(got, want, rtol=0.0, atol=0.0, equal_nan=True) & ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got - want)[bad].abs().max()),
                           float(torch.as_tensor(tol, device=got.device).expand_as(got)[bad].min()))


def check_grads(c, out, ref, scale=1.0, base=None, grad="same", moves=0.0):
    """ref: seq_ref's outputs; scale: grad_scale; base: what was in the gradients before (accumulation)."""
    slope = ref["slope"] * scale
    x = torch.where(c.on[:, None], c.x, 0.0)
    g, a = R.grad_logits(x, torch.where(c.on, c.targets, 0), c.on, slope, c.T)
    p = torch.where(c.on[:, None], torch.softmax(x, -1), 0.0)
    # what an element's coefficient and probability are rounded and moved relative to
    mass = ref["mass"] * abs(scale) / c.T
    size, own = mass[:, None] * p, a.abs()[:, None] * p
    rows = torch.nonzero(c.on)[:, 0]
    size[rows, c.targets[rows]] += mass[rows]
    own[rows, c.targets[rows]] += a.abs()[rows]
    rel = 8.0 * c.lp_tol() + moves + 2.0 ** -20
    half = HALF[c.dtype]
    # fp32 and bf16 end at 2^-126: a probability, its product with the coefficient and a result below it may be zero
    under = 2.0 ** -126 * (2.0 + float(a.abs().max()))
    if not c.d:
        want = g if base is None else g + base.double()
        close(out["grad_logits"], want, rel * size + half * want.abs() + TINY[c.dtype] + under, "grad_logits")
        return
    h, w = torch.where(c.on[:, None], c.hidden.double(), 0.0), c.weight.double()
    # fp16 tiles hold the coefficients scaled to 2^14: their smallest step is 2^-39 of the largest
    tile = 0.0 if c.dtype == "f32" else half
    sums = rel + (c.d + max(c.n, c.V) / 16) * 2.0 ** -23
    fine = 2.0 ** -38 * float(a.abs().max()) if c.dtype == "f16" else 0.0
    out_half = half if grad == "same" and c.dtype != "f32" else 2.0 ** -24
    tiny = (TINY[c.dtype] if grad == "same" else 0.0) + 2.0 ** -126
    err = tile * own + sums * size + fine + under
    for name, m, ab in (("d_hidden", g @ w, err @ w.abs()), ("d_weight", g.t() @ h, err.t() @ h.abs())):
        if out[name] is None:
            continue
        want = m if base is None else m + base[name].double()
        close(out[name], want, ab + out_half * want.abs() + tiny, name)


def run_policy(c, flags=0, kl=0.0, low=0.2, high=0.2, **kw):
    given = (c.hidden, c.weight) if c.d else (c.logits,)
    f = L.lossk_policy_fwd_bwd if c.d else L.lossk_policy_from_logits
    return f(*given, c.targets, c.adv if not flags & L.SEQ_ADVANTAGES else c.seq_adv, c.old, c.ref, c.first, c.mask, low,
             high, kl, c.T, flags=flags, **kw)


def check_policy(c, out, flags=0, kl=0.0, low=0.2, high=0.2, scale=1.0, old=True, ref=True, **kw):
    adv = c.seq_adv if flags & L.SEQ_ADVANTAGES else c.adv
    r = R.policy(c.lp, c.on, c.first, adv, c.old if old else None, c.ref if ref else None, low, high, kl,
                 bool(flags & L.SEQ_RATIO), bool(flags & L.SEQ_MEAN), bool(flags & L.SEQ_ADVANTAGES),
                 bool(flags & L.REDUCE_SUM))
    tol = c.lp_tol()
    close(out["logp"], r["logp"], tol + 2.0 ** -24 * r["logp"].abs(), "logp")
    # |dL / dlogp| is at most ratio * |A| + kl * e^|q|
    live = c.on & torch.isfinite(adv if not flags & L.SEQ_ADVANTAGES else c.adv.nan_to_num(posinf=0, neginf=0))
    big = float((adv[c.on] if not flags & L.SEQ_ADVANTAGES else adv).abs().max()) if live.any() else 0.0
    lip = 2.0 * big + kl * 12.0
    close(out["per_token"], r["per_token"], tol * lip + 2.0 ** -21 * (r["per_token"].abs() + big), "per_token")
    weight = float(c.on.sum()) if flags & L.REDUCE_SUM else 1.0
    bound = torch.tensor([lip, 2.0 * big, 12.0, 1.0], device="cuda", dtype=torch.float64)
    close(out["scalars"], r["scalars"], weight * (tol + 2.0 ** -21) * (bound + 1.0) + 2.0 ** -22 * r["scalars"].abs(), "scalars")
    check_grads(c, out, r, scale, **kw)
    return r


def run_preference(c, flags=0, **kw):
    given = (c.hidden, c.weight) if c.d else (c.logits,)
    f = L.lossk_preference_fwd_bwd if c.d else L.lossk_preference_from_logits
    return f(*given, c.targets, c.first, c.ref, c.mask, flags=flags, **kw)


def check_preference(c, out, flags=0, scale=1.0, grads=True, **kw):
    opts = {k: kw.pop(k) for k in ("objective", "beta", "margin", "smoothing", "nll") if k in kw}
    r = R.preference(c.lp, c.on, c.first, c.ref, length_mean=bool(flags & L.LENGTH_MEAN), summed=bool(flags & L.REDUCE_SUM),
                     **opts)
    tol, beta = c.lp_tol(), opts.get("beta", 0.1)
    longest = max(len(g) for g in R.groups(c.n, c.first, c.on))
    many = 1 if flags & L.LENGTH_MEAN else max(1, longest)
    close(out["logp"], r["logp"], tol + 2.0 ** -24 * r["logp"].abs(), "logp")
    size = 2.0 ** -24 * (r["logp"].abs().max() + 1.0)
    far = many * (tol + size)                              # of a sequence's log ratio
    close(out["log_ratio"], r["log_ratio"], far + 2.0 ** -23 * r["log_ratio"].abs(), "log_ratio")
    u = float((r["log_ratio"][:len(r["per_pair"])] - r["log_ratio"][len(r["per_pair"]):]).abs().max())
    lip = 2.0 * (u + 0.5 / beta) + 1.0 if opts.get("objective") == "squared" else beta
    close(out["per_pair"], r["per_pair"], 2 * far * lip + 2.0 ** -21 * (1.0 + r["per_pair"].abs()), "per_pair")
    pairs = len(r["per_pair"]) if flags & L.REDUCE_SUM else 1
    toks = int(c.on.sum()) if flags & L.REDUCE_SUM else 1
    nll = opts.get("nll", 0.0)
    size_l = toks * (tol + size)
    bound = torch.tensor([pairs * 2 * far * lip + nll * size_l, pairs * 2 * far * lip, size_l, 0.0], device="cuda",
                         dtype=torch.float64)
    close(out["scalars"], r["scalars"], bound + 2.0 ** -21 * (1.0 + r["scalars"].abs()), "scalars")
    if grads:
        check_grads(c, out, r, scale, moves=4.0 * beta * far, **kw)
    return r


LOGITS = [(1, 1, "f32", {}), (1, 7, "bf16", {}), (3, 129, "f16", {}), (37, 1000, "bf16", dict(masked=0.3)),
          (64, 4099, "f32", dict(seqs=5, masked=0.2, tail=3)), (130, 12289, "f16", dict(seqs=9, empty=True, T=0.7)),
          (257, 2051, "bf16", dict(seqs=3, masked=0.5, T=1.4)), (9, 40000, "bf16", dict(seqs=2)),
          (700, 515, "bf16", dict(masked=0.1))]
HEAD = [(1, 8, 8, "bf16", {}), (5, 1, 16, "bf16", {}), (64, 1000, 64, "f32", dict(masked=0.2)),
        (37, 1030, 72, "f16", dict(seqs=4, masked=0.3)), (130, 515, 264, "bf16", dict(seqs=5, tail=7, empty=True)),
        (300, 2000, 320, "bf16", dict(seqs=6, masked=0.4, T=0.8)), (257, 777, 128, "f16", dict(masked=0.1, T=1.3)),
        (33, 300, 20, "f32", dict(seqs=3, T=0.9)), (512, 4096, 1024, "bf16", dict(seqs=8))]


def make(size, **kw):
    if len(size) == 4:
        n, V, dtype, opts = size
        return Case(n, V, dtype, **{**opts, **kw})
    n, V, d, dtype, opts = size
    return Case(n, V, dtype, d=d, **{**opts, **kw})


@pytest.mark.parametrize("size", LOGITS + HEAD, ids=str)
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_policy_by_token(size, kl):
    c = make(size)
    kw = dict(grad_dtype=DT[c.dtype]) if c.d else {}
    check_policy(c, run_policy(c, kl=kl, grad_scale=1.5, **kw), kl=kl, scale=1.5)


@pytest.mark.parametrize("size", [s for s in LOGITS + HEAD if s[-1].get("seqs")], ids=str)
@pytest.mark.parametrize("flags", [L.SEQ_RATIO, L.SEQ_MEAN, L.SEQ_RATIO | L.SEQ_MEAN | L.SEQ_ADVANTAGES,
                                   L.SEQ_ADVANTAGES | L.REDUCE_SUM, L.SEQ_MEAN | L.REDUCE_SUM])
def test_policy_by_sequence(size, flags):
    c = make(size)
    c.seq_adv = torch.randn(len(c.first) - 1, device="cuda", generator=gen(3))
    kw = dict(grad_dtype=DT[c.dtype]) if c.d else {}
    check_policy(c, run_policy(c, flags, kl=0.05, low=0.013, high=0.017, **kw), flags, kl=0.05, low=0.013, high=0.017)


@pytest.mark.parametrize("size", [LOGITS[4], HEAD[3], HEAD[4]], ids=str)
def test_policy_without_old_or_reference(size):
    c = make(size)
    given = (c.hidden, c.weight) if c.d else (c.logits,)
    f = L.lossk_policy_fwd_bwd if c.d else L.lossk_policy_from_logits
    out = f(*given, c.targets, c.adv, first=c.first, loss_mask=c.mask, temperature=c.T)
    check_policy(c, out, old=False, ref=False, **(dict(grad="float") if c.d else {}))


PAIRS = [(40, 700, "bf16", dict(seqs=4, masked=0.2)), (130, 4099, "f16", dict(seqs=6, tail=5, empty=True)),
         (64, 1000, "f32", dict(seqs=2)), (2, 3, "f32", dict(seqs=2)), (300, 1031, "bf16", dict(seqs=64)),
         (130, 515, 264, "bf16", dict(seqs=4, masked=0.3)), (64, 1000, 64, "f32", dict(seqs=4)),
         (203, 1200, 136, "f16", dict(seqs=6, masked=0.2, tail=9))]


@pytest.mark.parametrize("size", PAIRS, ids=str)
@pytest.mark.parametrize("opts", [dict(), dict(margin=0.4, smoothing=0.2, beta=0.3), dict(objective="hinge", beta=0.2),
                                  dict(objective="squared", beta=0.5), dict(nll=0.7)], ids=str)
@pytest.mark.parametrize("flags", [0, L.LENGTH_MEAN, L.REDUCE_SUM])
def test_preference(size, opts, flags):
    c = make(size)
    kw = dict(opts)
    if "smoothing" in kw:
        kw["label_smoothing"] = kw.pop("smoothing")
    if "nll" in kw:
        kw["nll_weight"] = kw.pop("nll")
    if c.d:
        kw["grad_dtype"] = DT[c.dtype]
    check_preference(c, run_preference(c, flags, **kw), flags, **opts)
