"""The policy and preference losses where coefficients are of very different sizes, one of them is no number, or all are far
from 1: what a row gets depends on its own coefficient alone."""
import math

import pytest
import torch

import output_projection_cross_gb300 as L
import seq_ref as R
from test_gpu_sequence import (DT, HALF, TINY, Case, check_grads, check_policy, check_preference, close, run_policy,
                               run_preference)

pytestmark = pytest.mark.gpu
HEADS = [dict(n=70, V=900, d=136, dtype="f16"), dict(n=300, V=2001, d=264, dtype="f16"), dict(n=70, V=900, d=136, dtype="bf16"),
         dict(n=70, V=900, d=72, dtype="f32")]


def check_rows(c, out, rows, scale, grad, adv):
    """d_hidden of `rows` against the 64-bit definition; each row's error is relative to its own coefficient."""
    r = R.policy(c.lp, c.on, c.first, adv, c.old, c.ref)
    g, a = R.grad_logits(c.x, c.targets, c.on, r["slope"] * scale, c.T)
    p = torch.softmax(c.x, -1)
    mass = r["mass"] * scale / c.T
    size, own = mass[:, None] * p, a.abs()[:, None] * p
    at = torch.arange(c.n)
    size[at, c.targets] += mass
    own[at, c.targets] += a.abs()
    half = HALF[c.dtype]
    # as in test_gpu_sequence.check_grads, but that a row's tile ends 2^-38 below its own coefficient
    err = (0.0 if c.dtype == "f32" else half) * own + (8 * c.lp_tol() + 2.0 ** -20 + (c.d + c.V / 16) * 2.0 ** -23) * size
    err = err + (2.0 ** -38 * a.abs()[:, None] if c.dtype == "f16" else 0.0) + 2.0 ** -126 * (2.0 + a.abs()[:, None])
    w = c.weight.double()
    want = g @ w
    out_half = half if grad == "same" and c.dtype != "f32" else 2.0 ** -24
    tol = err @ w.abs() + out_half * want.abs() + (TINY[c.dtype] if grad == "same" else 0.0) + 2.0 ** -126
    close(out["d_hidden"][rows], want[rows], tol[rows], "d_hidden")


@pytest.mark.parametrize("kw", HEADS, ids=str)
@pytest.mark.parametrize("grad", ["same", "float"])
@pytest.mark.parametrize("what", ["hidden NaN", "hidden infinite", "ratio infinite", "ratio far above", "advantages"])
def test_one_row_costs_the_others_nothing(kw, grad, what):
    c = Case(**kw)
    rows = torch.ones(c.n, dtype=torch.bool, device="cuda")
    rows[5] = False
    # mean-reduced coefficients of a long batch
    scale = 1e-3
    if what == "hidden NaN":
        c.hidden[5] = math.nan
    elif what == "hidden infinite":
        c.hidden[5, 0] = math.inf
    elif what == "ratio infinite":
        c.old[5], c.adv[5] = float(c.lp[5]) - 200.0, -1.0
    elif what == "ratio far above":
        c.old[5], c.adv[5] = float(c.lp[5]) - 40.0, -1.0
    else:
        # sizes over 20 powers of ten, among them one that takes no part
        c.adv *= 10.0 ** torch.linspace(-12.0, 8.0, c.n, device="cuda")
        c.adv[5] = 0.0
    out = run_policy(c, grad_scale=scale, grad_dtype=DT[c.dtype] if grad == "same" else torch.float32)
    adv = c.adv.clone()
    if what.startswith("hidden"):
        c.x[5] = 0.0                                       # (the definition's row, left out of the comparison)
        c.lp = torch.where(rows, c.lp, 0.0)
    elif what.startswith("ratio"):
        adv[5] = 0.0
        assert not torch.isfinite(out["d_hidden"][5]).all() or what.endswith("above")
    check_rows(c, out, rows, scale, grad, adv)
    if what.startswith("hidden"):
        assert torch.isnan(out["logp"][5]) and torch.isfinite(out["logp"][rows]).all()


@pytest.mark.parametrize("kw", [dict(n=70, V=9000, dtype="f16"), dict(n=70, V=900, dtype="f16"), dict(n=70, V=9000, dtype="bf16"),
                                dict(n=70, V=9001, dtype="f32"), dict(n=9, V=500003, dtype="bf16")], ids=str)
@pytest.mark.parametrize("loss", ["policy", "pairs"])
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e3, 1e20])
def test_scales_of_given_logits_gradient(kw, loss, scale):
    """The gradient has the scale, and what its type does not hold of it is 0 or infinite; nothing else moves."""
    c = Case(seqs=2, masked=0.2, **kw)
    run, kwargs = (run_policy, dict(kl=0.1)) if loss == "policy" else (run_preference, {})
    one, out = run(c, **kwargs), run(c, grad_scale=scale, **kwargs)
    for k in one:
        if k != "grad_logits":
            assert torch.equal(one[k], out[k]), k
    (check_policy if loss == "policy" else check_preference)(c, one, **kwargs)
    g = out["grad_logits"]
    assert not torch.isnan(g).any() and not g[~c.on].any()
    if c.dtype == "f16" and scale == 1e-30:
        assert not g.any()                                 # below fp16's smallest, 6e-8
        return
    if c.dtype == "f16" and scale == 1e20:
        assert torch.isinf(g).any()                        # above its largest, 65504
        return
    r = (R.policy(c.lp, c.on, c.first, c.adv, c.old, c.ref, kl=0.1) if loss == "policy"
         else R.preference(c.lp, c.on, c.first, c.ref))
    moves = 0.0 if loss == "policy" else 4.0 * 0.1 * max(len(s) for s in R.groups(c.n, c.first, c.on)) * (
        c.lp_tol() + 2.0 ** -24 * (float(r["logp"].abs().max()) + 1.0))
    check_grads(c, out, r, scale=scale, moves=moves)
    assert g[c.on].any()
