"""The policy and preference losses from given logits whose values lie far out: masks of the type's lowest value, a common
offset, temperatures far below 1.

Tolerances of a gradient element, where the coefficient is exact: the distance to the row's largest logit and its product
with the scale are rounded once each (2^-23 of an argument of at most 64 where the probability is above 2^-64: 64 ln 2
2^-23), the row's sum as in test_gpu_sequence (4e-6 of additions, 2^-21 of ex2.approx), the result to its type."""
import math

import pytest
import torch

import output_projection_cross_gb300 as L
import seq_ref as R
from test_gpu_sequence import DT, HALF, TINY, Case, check_policy, check_preference, close, gen, run_policy, run_preference

pytestmark = pytest.mark.gpu
REL = 64.0 * 2.0 ** -23 + 4e-6 + 2.0 ** -21

# a warp's rows, a cluster's, and rows too long for it
ROWS = [dict(n=40, V=900, dtype="bf16"), dict(n=40, V=901, dtype="f32"), dict(n=40, V=9001, dtype="bf16"),
        dict(n=24, V=9001, dtype="f32"), dict(n=16, V=9001, dtype="f16"), dict(n=24, V=100003, dtype="bf16"),
        dict(n=400, V=40003, dtype="f32"), dict(n=6, V=500003, dtype="bf16")]


def shifted(c):
    """The case's scaled logits, each row's largest at 0 (in double their sums lose nothing then)."""
    x = c.logits.double()
    return (x - x.max(1, keepdim=True).values) / c.T


@pytest.mark.parametrize("kw", ROWS, ids=str)
@pytest.mark.parametrize("by", ["token", "sequence", "pair"])
def test_masks_of_the_lowest_value(kw, by):
    c = Case(seqs=4, **kw)
    g, low = gen(5), torch.finfo(DT[c.dtype]).min
    hide = torch.rand(c.n, c.V, device="cuda", generator=g) < 0.3
    hide[: c.n // 2, : c.V // 2] = True                     # whole threads' and pieces' shares
    hide[:, -3:] = True
    hide[torch.arange(c.n), c.targets.clamp_(max=c.V - 4)] = False
    c.logits[hide] = low
    c.logits[3] = low                                       # a uniform row
    c.logits[4] = low
    c.logits[4, 5] = -math.inf
    c.targets[4] = 6
    c.x = shifted(c)
    c.fill(g)
    if by == "pair":
        check_preference(c, run_preference(c))
        return
    flags = L.SEQ_RATIO if by == "sequence" else 0
    band = dict(low=0.013, high=0.017) if flags else {}
    out = run_policy(c, flags, kl=0.1, **band)
    check_policy(c, out, flags, kl=0.1, **band)
    rest = torch.ones(c.n, dtype=torch.bool, device="cuda")
    rest[3:5] = False
    assert not out["grad_logits"][hide & rest[:, None]].any()


def exact_rows(c, out):
    """grad_logits of a policy gradient with advantages as coefficients."""
    p = torch.softmax(c.x, -1)
    g, a = R.grad_logits(c.x, c.targets, c.on, -c.adv.double(), c.T)
    own = a.abs()[:, None] * p
    hit = torch.zeros_like(own)
    hit[torch.arange(c.n), c.targets] = a.abs()
    under = 2.0 ** -126 * (2.0 + float(a.abs().max()))
    close(out["grad_logits"], g, REL * own + 2.0 ** -22 * (own + hit) + HALF[c.dtype] * g.abs() + TINY[c.dtype] + under, "grad_logits")


@pytest.mark.parametrize("kw", [r for r in ROWS if r["dtype"] == "f32"], ids=str)
@pytest.mark.parametrize("offset", [0.0, 30.0, -3000.0, 1e5])
def test_a_common_offset(kw, offset):
    """Every probability relative to its own size, whatever all logits have in common."""
    c = Case(**kw)
    c.logits += offset
    c.x = shifted(c)
    c.lp = R.logprobs(c.x, c.targets, c.on)
    # -A (total = -sum A logp): a_t = A_t
    out = L.lossk_policy_from_logits(c.logits, c.targets, c.adv, flags=L.REDUCE_SUM)
    close(out["logp"], c.lp, c.lp_tol() + 2.0 ** -24 * c.lp.abs(), "logp")
    exact_rows(c, out)
    first = torch.tensor([0, c.n // 2, c.n], dtype=torch.int32, device="cuda")
    c.first, c.ref = first, c.lp.float()
    out = run_preference(c)
    # The reference's log-probabilities are the rounded exact ones, so u is the difference of two sums of roundings, each
    # below its tolerance: whether it is above 0 is open, and the share of such pairs 0 or 1.
    assert float(out["scalars"][3]) in (0.0, 1.0)
    out["scalars"][3] = R.preference(c.lp, c.on, c.first, c.ref)["scalars"][3]
    check_preference(c, out)


@pytest.mark.parametrize("kw", ROWS, ids=str)
@pytest.mark.parametrize("T", [1e-6, 1e-9, 1e-20, 1e-30, 1e30])
def test_temperatures_far_from_one(kw, T):
    """Where logits over the temperature differ by less than fp32's range in log2 units or by far more."""
    c = Case(**kw)
    c.T = T
    rows = torch.arange(c.n, device="cuda")
    near = rows < c.n // 2
    c.targets = torch.where(near, c.logits.float().argmax(1), c.targets)
    c.x = shifted(c)
    c.lp = R.logprobs(c.x, c.targets, c.on)
    out = L.lossk_policy_from_logits(c.logits, c.targets, c.adv, temperature=T, flags=L.REDUCE_SUM, grad_scale=min(T, 1.0))
    assert not torch.isnan(out["logp"]).any() and not torch.isnan(out["grad_logits"]).any()
    far = c.lp.float().double()                             # -infinity beyond fp32
    close(out["logp"], torch.where(torch.isinf(far), far, c.lp), 8e-6 + 2.0 ** -22 * c.lp.abs(), "logp")
    c.adv *= min(T, 1.0)
    exact_rows(c, out)


def exact_head(offset, T=1.0, V=1001):
    """One token in fp32 and a head whose logits are exact sums: hidden, weight, target, scaled logits (the largest 0)."""
    hidden = torch.tensor([[1.0, 1.0]], device="cuda")
    weight = torch.stack([torch.randint(-2048, 2049, (V,), device="cuda", generator=gen(3)) / 256.0,
                          torch.full((V,), offset, device="cuda")], 1).contiguous()
    x = hidden.double() @ weight.double().t()
    assert torch.equal(x, x.float().double())
    return hidden, weight, torch.tensor([7], device="cuda"), (x - x.max()) / T


@pytest.mark.parametrize("offset", [0.0, 48.0, 300.0, 3000.0, -20000.0])
@pytest.mark.parametrize("T", [1.0, 0.7, 1.3])
def test_logp_of_a_head_with_a_common_offset(offset, T):
    hidden, weight, y, x = exact_head(offset, T)
    out = L.lossk_policy_fwd_bwd(hidden, weight, y, torch.ones(1, device="cuda"), temperature=T)
    want = torch.log_softmax(x, -1)[:, 7]
    # as from given logits, and the scale's two roundings (2^-23 of a distance to the target's logit)
    close(out["logp"], want, 8e-6 + 2.0 ** -22 * want.abs(), "logp")


@pytest.mark.parametrize("offset", [0.0, 48.0, 3000.0, -20000.0])
def test_gradient_of_a_head_with_a_common_offset(offset):
    """d_weight's first column is a p_v (a - a p_y the target's)."""
    hidden, weight, y, x = exact_head(offset)
    out = L.lossk_policy_fwd_bwd(hidden, weight, y, torch.ones(1, device="cuda"))
    p = torch.softmax(x, -1)[0]
    hit = torch.arange(len(p), device="cuda") == 7
    want = p - hit.double()
    # one rounding of an argument below 32 (32 ln 2 2^-24), exp2f's two units, the row's sum (test_gpu_sequence)
    tol = (32 * 2.0 ** -24 + 2.0 ** -22 + 4e-6) * (p + hit * p[7]) + 2.0 ** -24 * want.abs()
    close(out["d_weight"][:, 0], want, tol, "d_weight")


@pytest.mark.parametrize("kw", ROWS + [dict(n=40, V=1, dtype=t) for t in ("bf16", "f16", "f32")], ids=str)
@pytest.mark.parametrize("loss", ["policy", "pairs"])
def test_a_certain_token_has_logp_0(kw, loss):
    """All but the target 40 below it and more: its sum is 1 to the last bit, and so is its probability."""
    c = Case(**kw)
    c.logits.clamp_(-20.0, 20.0)
    c.logits[torch.arange(c.n), c.targets] = 60.0
    if loss == "policy":
        out = L.lossk_policy_from_logits(c.logits, c.targets, c.adv)
    else:
        out = L.lossk_preference_from_logits(c.logits, c.targets, torch.tensor([0, c.n // 2, c.n], dtype=torch.int32, device="cuda"))
    assert not out["logp"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 300])
def test_certain_tokens_of_a_head(dtype, V):
    """logp without a bias: a sum about 1 is rounded by 2^-24 at most, up in some rows and down in others."""
    n, d = 1000, 64
    c = Case(n=n, V=V, d=d, dtype=dtype, std=0.2)
    c.hidden[:, :2] = 0.0
    c.hidden[:, 0] = 8.0
    c.weight[:, 0] = 0.0
    c.weight[0, 0] = 6.0
    c.targets.zero_()
    out = L.lossk_policy_fwd_bwd(c.hidden, c.weight, c.targets, c.adv, want_d_hidden=False, want_d_weight=False)
    assert abs(float(out["logp"].double().mean())) <= 2.0 ** -24 and float(out["logp"].abs().max()) <= 2.0 ** -21


@pytest.mark.parametrize("kw", [dict(n=9, V=900, dtype="bf16"), dict(n=9, V=9001, dtype="f32"), dict(n=3, V=500003, dtype="bf16")], ids=str)
@pytest.mark.parametrize("flags", [0, L.SEQ_MEAN, L.SEQ_RATIO])
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_kl_of_a_token_of_probability_0(kw, flags, kl):
    """exp(q) - q - 1 of an infinite q is infinite, and so is what it is part of; without a weight it stays out of the total."""
    c = Case(seqs=2, **kw)
    c.logits[1, c.targets[1]] = -math.inf
    c.adv.abs_()
    c.x = c.logits.double()
    c.lp = R.logprobs(c.x, c.targets, c.on)
    c.old[1], c.ref[1] = -8.0, -9.0
    out = run_policy(c, flags, kl=kl)
    total, policy, far = (float(v) for v in out["scalars"][:3])
    assert math.isinf(float(out["logp"][1])) and far == math.inf and math.isfinite(policy)
    assert total == (math.inf if kl else policy)
    rest = torch.arange(c.n, device="cuda") != 1
    assert torch.isfinite(out["per_token"][rest]).all()
    if not flags & L.SEQ_RATIO:
        assert float(out["per_token"][1]) == (math.inf if kl else 0.0)


@pytest.mark.parametrize("kw", [dict(n=40, V=900, dtype="f32"), dict(n=24, V=9001, dtype="f32")], ids=str)
@pytest.mark.parametrize("T,scale", [(1e-20, 1e25), (1e-30, 1e9), (1e30, 1e-30)])
def test_a_scale_over_the_temperature_beyond_floats(kw, T, scale):
    """1e39 and more, or nothing: a token without an advantage has a zero gradient, one with a small one a finite one."""
    c = Case(**kw)
    c.T = T
    c.adv *= 1e-35 if scale > 1.0 else 1e35
    c.adv[::2] = 0.0
    c.x = shifted(c)
    out = L.lossk_policy_from_logits(c.logits, c.targets, c.adv, temperature=T, grad_scale=scale, flags=L.REDUCE_SUM)
    assert not out["grad_logits"][::2].any()
    assert T > 1.0 or out["grad_logits"][1::2].any()
    c.adv = c.adv.double() * scale
    exact_rows(c, out)


@pytest.mark.parametrize("kw", [dict(n=40, V=900, d=136, dtype="bf16"), dict(n=40, V=900, d=136, dtype="f16"), dict(n=40, V=900, d=72, dtype="f32")],
                         ids=str)
@pytest.mark.parametrize("T", [1e-3, 1e-5, 1e-7, 1e-9, 1e-20, 1e-30])
@pytest.mark.parametrize("forward", [False, True])
def test_a_head_at_temperatures_far_below_one(kw, T, forward):
    """logp as far off as the logits over the temperature are, and no number where its log-sum-exp passes 7e8."""
    c = Case(**kw)
    s = c.x
    c.T, c.x = T, (s - s.max(1, keepdim=True).values) / T
    want = R.logprobs(c.x, c.targets, c.on)
    lse = s.max(1).values / T
    assert float(lse.min()) > 7.5e8 or float(lse.max()) < 7.3e8
    kwargs = dict(want_d_hidden=False, want_d_weight=False) if forward else {}
    out = L.lossk_policy_fwd_bwd(c.hidden, c.weight, c.targets, c.adv, temperature=T, grad_scale=T, **kwargs)
    if float(lse.min()) > 7.5e8:
        assert torch.isnan(out["logp"]).all()
        return
    # a logit's error in test_gpu_sequence's lp_tol, and the scale's rounding
    top = float(s.abs().max())
    sums = 2.0 ** -22 if c.dtype == "f32" else (c.d / 16 + 8) * 2.0 ** -22
    close(out["logp"], want, 8e-6 + (sums + 2.0 ** -22) * top / T, "logp")
    if not forward:
        assert torch.isfinite(out["d_hidden"]).all() and torch.isfinite(out["d_weight"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [1024, 4096])
@pytest.mark.parametrize("how", ["even", "few large", "first", "last", "falling"])
def test_what_the_tensor_cores_drop(dtype, d, how):
    """How far logits are off in proportion to their size, by how their sums grow along d_model.

    A step of 16 products drops half of a sum's last bit on average, 2^-24 of it or less (0.72 of that over a binade), so a
    logit comes out low by 0 to 0.72 * 2^-24 / 16 = 2.7e-9 of itself per unit of d_model.  The passes scale 1e-9 of that
    back for every row, whatever its sums are like: between 1.7e-9 low and 1e-9 high is left (and 1e-10 of noise)."""
    g, n, V = gen(11), 512, 8000
    h = torch.randn(n, d, device="cuda", generator=g)
    if how == "few large":
        h[:, torch.randperm(d, device="cuda", generator=g)[:8]] *= 40.0
    elif how in ("first", "last"):
        h[:, 0 if how == "first" else -1] *= 200.0
    elif how == "falling":
        h *= torch.logspace(1.0, -1.0, d, device="cuda")
    hidden = (h / h.pow(2).mean(1, keepdim=True).sqrt()).to(DT[dtype])
    weight = (torch.randn(V, d, device="cuda", generator=g) * (2.5 / math.sqrt(d))).to(DT[dtype])
    x = hidden.double() @ weight.double().t()
    p = torch.softmax(x, -1)
    y = torch.multinomial(p, 1, generator=g)[:, 0]
    rows = torch.arange(n, device="cuda")
    out = L.lossk_policy_fwd_bwd(hidden, weight, y, torch.ones(n, device="cuda"), want_d_hidden=False, want_d_weight=False)
    off = out["logp"].double() - torch.log_softmax(x, -1)[rows, y]
    # logits of 1 + e times their size move logp by e (x_y - E x)
    lever = x[rows, y] - (p * x).sum(1)
    e = float((off * lever).sum() / lever.pow(2).sum()) / d
    print(how, e)
    assert -1.8e-9 < e < 1.1e-9
