"""The policy and preference losses where they can go wrong: nothing that counts, masked vocabularies, rows that the fused
pass cannot represent, wrong targets and sequences, gradients added and written in place, graphs, streams, a workspace
used for one call after another, logits of more than 2^31 elements."""
import math
import os
import subprocess
import sys

import pytest
import torch

import output_projection_cross_gb300 as L
import seq_ref as R
from test_gpu_sequence import (CODE, DT, Case, check_grads, check_policy, check_preference, close, gen, run_policy,
                               run_preference)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADS = [dict(n=70, V=900, d=136, dtype="bf16"), dict(n=70, V=900, d=136, dtype="f16"), dict(n=70, V=900, d=72, dtype="f32")]
ROWS = [dict(n=70, V=900, dtype="bf16"), dict(n=40, V=9001, dtype="f16"), dict(n=40, V=9001, dtype="f32"),
        dict(n=33, V=20011, dtype="bf16")]


def of(c):
    return dict(grad_dtype=DT[c.dtype]) if c.d else {}


def grads_of(out):
    return [out[k] for k in ("d_hidden", "d_weight", "grad_logits") if out.get(k) is not None]


@pytest.mark.parametrize("kw", HEADS + ROWS, ids=str)
@pytest.mark.parametrize("how", ["mask", "sequences"])
def test_nothing_counts(kw, how):
    c = Case(seqs=2 if how == "sequences" else 0, **kw)
    if how == "mask":
        c.mask = torch.zeros(c.n, dtype=torch.uint8, device="cuda")
    else:
        c.first = torch.tensor([5, 5, 5], dtype=torch.int32, device="cuda")
    c.targets.fill_(-1)
    given = (c.hidden, c.weight) if c.d else (c.logits,)
    f = L.lossk_policy_fwd_bwd if c.d else L.lossk_policy_from_logits
    ws = L.sequence_workspace(0 if c.d else 1, c.n, max(c.d, 1), c.V, 2, CODE[c.dtype])
    outs = [f(*given, c.targets, c.adv, c.old, c.ref, c.first, c.mask, kl_weight=0.1, ws=ws, **of(c))]
    if how == "sequences":
        g = L.lossk_preference_fwd_bwd if c.d else L.lossk_preference_from_logits
        outs.append(g(*given, c.targets, c.first, c.ref, c.mask, nll_weight=1.0, ws=ws, **of(c)))
    for out in outs:
        for k, v in out.items():
            assert v is None or not v.any(), k
    assert L.lossk_device_status(ws) == 580


@pytest.mark.parametrize("kw", ROWS, ids=str)
@pytest.mark.parametrize("by", ["token", "sequence", "pair"])
def test_masked_vocabulary(kw, by):
    """Entries at -infinity have probability 0; a row of nothing else has logp -infinity and a zero gradient."""
    c = Case(seqs=4, **kw)
    g = gen(5)
    hide = torch.rand(c.n, c.V, device="cuda", generator=g) < 0.4
    hide[torch.arange(c.n, device="cuda"), c.targets] = False
    c.logits[hide] = -math.inf
    c.logits[:, -3:] = -math.inf                            # a row's last vector
    c.targets.clamp_(max=c.V - 4)
    c.logits[torch.arange(c.n, device="cuda"), c.targets] = 1.0
    c.logits[7] = -math.inf
    c.x = c.logits.double()
    c.fill(g)
    keep = c.on.clone()
    c.old[7], c.ref[7] = 0.0, 0.0
    assert torch.isneginf(c.lp[7])
    if by == "pair":
        # an infinitely unlikely sequence: its pair is left out of the comparison here
        c.mask = keep.to(torch.uint8)
        c.mask[7] = 0
        c.on = keep & (c.mask != 0)
        c.lp = R.logprobs(c.x, c.targets, c.on)
        check_preference(c, run_preference(c))
        return
    flags = L.SEQ_RATIO if by == "sequence" else 0
    out = run_policy(c, flags)
    r = R.policy(c.lp, c.on, c.first, c.adv, c.old, c.ref, seq_ratio=bool(flags))
    close(out["logp"], r["logp"], 1e-5, "logp")
    assert not out["grad_logits"][7].any()
    assert not out["grad_logits"][hide].any()
    live = torch.ones(c.n, dtype=torch.bool, device="cuda")
    live[7] = False
    if by == "token":
        close(out["per_token"][live], r["per_token"][live], 1e-4, "per_token")


def test_a_nan_stays_in_its_row():
    c = Case(n=20, V=5000, dtype="bf16")
    c.logits[3, 4999] = math.nan
    c.logits[4] = -math.inf
    c.logits[4, 17] = math.nan
    out = run_policy(c)
    assert torch.isnan(out["logp"][[3, 4]]).all() and torch.isnan(out["grad_logits"][[3, 4]]).any(1).all()
    rest = [i for i in range(20) if i not in (3, 4)]
    assert torch.isfinite(out["logp"][rest]).all() and torch.isfinite(out["grad_logits"][rest]).all()


def far_target(d=64, gap=200.0):
    """Rows whose target lies `gap` below their largest logit: beyond what the fused pass's reference covers."""
    c = Case(n=40, V=600, d=d, dtype="bf16", std=0.5)
    c.hidden[:, 0] = 4.0
    c.weight[:, 0] = 0.0
    c.weight[5, 0] = gap / 4.0
    c.hidden[20:, 0] = 0.0                                   # the other half stays ordinary
    c.x = c.hidden.double() @ c.weight.double().t()
    c.targets.clamp_(min=6)
    c.fill(gen(2))
    return c


@pytest.mark.parametrize("grad", ["same", "float", "added"])
def test_rows_beyond_the_fused_pass(grad):
    c = far_target()
    flags, kw, base = 0, dict(grad_dtype=DT[c.dtype]), None
    if grad != "same":
        kw = dict(grad_dtype=torch.float32)
    if grad == "added":
        g = gen(9)
        base = dict(d_hidden=torch.randn(c.n, c.d, device="cuda", generator=g),
                    d_weight=torch.randn(c.V, c.d, device="cuda", generator=g))
        kw = {k: v.clone() for k, v in base.items()}
        flags = L.ACCUMULATE_GRADS
    out = run_policy(c, flags, kl=0.0, **kw)
    r = R.policy(c.lp, c.on, c.first, c.adv, c.old, c.ref)
    close(out["logp"], r["logp"], c.lp_tol() + 2.0 ** -23 * r["logp"].abs(), "logp")
    check_grads(c, out, r, base=base, grad="same" if grad == "same" else "float", moves=1e-4)


def test_a_sum_beyond_floats():
    """Weights near fp32's end: d_hidden's shifted sum overflows, the true one does not."""
    c = Case(n=8, V=300, d=64, dtype="bf16", std=0.5)
    c.hidden[:, 1] = 0.0
    c.weight[:, 1] = 1e33
    c.x = c.hidden.double() @ c.weight.double().t()
    c.fill(gen(3))
    out = run_policy(c, grad_dtype=torch.float32)
    r = R.policy(c.lp, c.on, None, c.adv, c.old, c.ref)
    assert torch.isfinite(out["d_hidden"]).all()
    g, a = R.grad_logits(c.x, c.targets, c.on, r["slope"])
    want = g @ c.weight.double()
    close(out["d_hidden"][:, 2:], want[:, 2:], 0.02 * float(a.abs().max()) * float(c.weight[:, 2:].abs().max()), "d_hidden")


@pytest.mark.parametrize("kw", HEADS + ROWS, ids=str)
def test_gradients_added(kw):
    """Into float gradients (hidden rows) or the logits' own type, with sums instead of means."""
    c = Case(seqs=4, masked=0.3, tail=5, **kw)
    g = gen(8)
    flags = L.ACCUMULATE_GRADS | L.REDUCE_SUM
    if c.d:
        base = dict(d_hidden=torch.randn(c.n, c.d, device="cuda", generator=g),
                    d_weight=torch.randn(c.V, c.d, device="cuda", generator=g))
    else:
        base = dict(grad_logits=torch.randn(c.n, c.V, device="cuda", generator=g).to(DT[c.dtype]))
    out = run_policy(c, flags, kl=0.05, **{k: v.clone() for k, v in base.items()})
    check_policy(c, out, flags, kl=0.05, base=base if c.d else base["grad_logits"], **(dict(grad="float") if c.d else {}))
    out = run_preference(c, flags, **{k: v.clone() for k, v in base.items()})
    check_preference(c, out, flags, base=base if c.d else base["grad_logits"], **(dict(grad="float") if c.d else {}))


@pytest.mark.parametrize("kw", HEADS, ids=str)
@pytest.mark.parametrize("want", [(False, False), (True, False), (False, True)])
def test_one_gradient_or_none(kw, want):
    c = Case(seqs=4, masked=0.2, **kw)
    kwargs = dict(want_d_hidden=want[0], want_d_weight=want[1], **of(c))
    out = run_policy(c, kl=0.1, **kwargs)
    assert (out["d_hidden"] is not None, out["d_weight"] is not None) == want
    check_policy(c, out, kl=0.1)
    check_preference(c, run_preference(c, **kwargs))


@pytest.mark.parametrize("kw", ROWS, ids=str)
def test_no_gradient_and_in_place(kw):
    c = Case(seqs=4, masked=0.2, **kw)
    c.seq_adv = c.adv[:4].nan_to_num(0.0, 0.0, 0.0).clone()
    for flags in (0, L.SEQ_RATIO | L.SEQ_ADVANTAGES):
        full = run_policy(c, flags)
        out = run_policy(c, flags, want_grad=False)
        assert out["grad_logits"] is None
        for k in ("scalars", "per_token", "logp"):
            assert torch.equal(out[k], full[k]), k
        keep = c.logits.clone()
        out = run_policy(c, flags, grad_logits=c.logits)
        assert torch.equal(out["grad_logits"], full["grad_logits"])
        c.logits.copy_(keep)
    full = run_preference(c)
    out = run_preference(c, grad_logits=c.logits)
    assert torch.equal(out["grad_logits"], full["grad_logits"])


@pytest.mark.parametrize("kw", HEADS + ROWS, ids=str)
@pytest.mark.parametrize("what", ["target", "negative", "first falls", "first past the end", "first negative"])
def test_wrong_device_data_is_refused(kw, what):
    c = Case(seqs=4, **kw)
    good = c.targets.clone(), c.first.clone()
    if what == "target":
        c.targets[c.n // 2] = c.V
    elif what == "negative":
        c.targets[c.n - 1] = -1
    else:
        c.first[{"first falls": 2, "first past the end": 4, "first negative": 0}[what]] = {
            "first falls": -(1 << 30), "first past the end": c.n + 1, "first negative": -1}[what]
    ws = L.sequence_workspace(0 if c.d else 1, c.n, max(c.d, 1), c.V, 4, CODE[c.dtype])
    mark = dict(scalars_out=torch.full((4,), 7.0, device="cuda"), logp_out=torch.full((c.n,), 7.0, device="cuda"))
    if c.d:
        mark.update(d_hidden=torch.full_like(c.hidden, 7.0), d_weight=torch.full_like(c.weight, 7.0))
    else:
        mark.update(grad_logits=torch.full_like(c.logits, 7.0))
    more = dict(per_token_out=torch.full((c.n,), 7.0, device="cuda"))
    pair = dict(per_pair_out=torch.full((2,), 7.0, device="cuda"), log_ratio_out=torch.full((4,), 7.0, device="cuda"))
    run_policy(c, ws=ws, **mark, **more)
    assert L.lossk_device_status(ws) == 586 and L.lossk_device_status(ws) == 580
    run_policy(c, L.SEQ_RATIO, ws=ws, **mark, **more)
    run_preference(c, ws=ws, **mark, **pair)
    assert L.lossk_device_status(ws) == 586
    for t in (*mark.values(), *more.values(), *pair.values()):
        assert (t == 7.0).all()
    # and the workspace serves the next call
    c.targets, c.first = good
    check_policy(c, run_policy(c, ws=ws, **of(c)))
    check_preference(c, run_preference(c, ws=ws, **of(c)))
    assert L.lossk_device_status(ws) == 580


def same(a, b):
    for k in a:
        if a[k] is not None:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


@pytest.mark.parametrize("kw", HEADS + ROWS, ids=str)
def test_bits_repeat(kw):
    c = Case(seqs=4, masked=0.2, tail=3, **kw)
    ws = L.sequence_workspace(0 if c.d else 1, c.n, max(c.d, 1), c.V, 4, CODE[c.dtype])
    a, b = run_policy(c, kl=0.1, **of(c)), run_preference(c, **of(c))
    for _ in range(3):
        same(a, run_policy(c, kl=0.1, ws=ws, **of(c)))
        same(b, run_preference(c, ws=ws, **of(c)))


@pytest.mark.parametrize("kw", HEADS + ROWS, ids=str)
def test_recorded_into_a_graph(kw):
    """Both losses in one graph, on one workspace, replayed on new inputs."""
    c, d = Case(seqs=4, masked=0.2, seed=1, **kw), Case(seqs=4, masked=0.2, seed=2, **kw)
    want = [(run_policy(x, kl=0.1, **of(x)), run_preference(x, **of(x))) for x in (c, d)]
    live = Case(seqs=4, masked=0.2, seed=3, **kw)
    ws = L.sequence_workspace(0 if c.d else 1, c.n, max(c.d, 1), c.V, 4, CODE[c.dtype])
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        a = run_policy(live, kl=0.1, ws=ws, **of(c))
        b = run_preference(live, ws=ws, **of(c))
    for x, (pa, pb) in zip((c, d, c), (want[0], want[1], want[0])):
        for k in ("hidden", "weight") if c.d else ("logits",):
            getattr(live, k).copy_(getattr(x, k))
        for k in ("targets", "first", "mask", "adv", "old", "ref"):
            getattr(live, k).copy_(getattr(x, k))
        graph.replay()
        torch.cuda.synchronize()
        same(pa, a)
        same(pb, b)
    assert L.lossk_device_status(ws) == 580


FIRST = """
import sys, torch
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import output_projection_cross_gb300 as L
from test_gpu_sequence import Case, DT, run_policy, run_preference
for kw in (dict(n=70, V=900, d=136, dtype="bf16"), dict(n=40, V=9001, dtype="f16")):
    c = Case(seqs=4, **kw)
    of = dict(grad_dtype=DT[c.dtype]) if c.d else {{}}
    ws = L.sequence_workspace(0 if c.d else 1, c.n, max(c.d, 1), c.V, 4, 1 if c.d else 2)
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        a = run_policy(c, ws=ws, **of)
        b = run_preference(c, ws=ws, **of)
    g.replay()
    torch.cuda.synchronize()
    for got, want in ((a, run_policy(c, **of)), (b, run_preference(c, **of))):
        for k in got:
            assert torch.equal(got[k], want[k]), k
    assert L.lossk_device_status(ws) == 580
print("recorded first")
"""


def test_first_calls_of_a_process_recorded():
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "recorded first" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("kw", [HEADS[0], HEADS[1], ROWS[1]], ids=str)
def test_on_another_stream(kw):
    """What is written on the call's own stream just before it is what it reads."""
    c, src = Case(seqs=4, seed=1, **kw), Case(seqs=4, seed=2, **kw)
    want = run_policy(src, **of(c)), run_preference(src, **of(c))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        for k in ("hidden", "weight") if c.d else ("logits",):
            getattr(c, k).copy_(getattr(src, k))
        for k in ("targets", "first", "adv", "old", "ref"):
            getattr(c, k).copy_(getattr(src, k))
    a, b = run_policy(c, stream=s, **of(c)), run_preference(c, stream=s, **of(c))
    s.synchronize()
    same(want[0], a)
    same(want[1], b)


def test_two_streams_at_once():
    """Calls on two streams with a workspace each, one after another without waiting."""
    cases = [Case(seqs=4, seed=i, **HEADS[0]) for i in (1, 2)] + [Case(seqs=4, seed=3, **ROWS[0])]
    want = [run_policy(c, **of(c)) for c in cases]
    ws = [L.sequence_workspace(0 if c.d else 1, c.n, max(c.d, 1), c.V, 4, CODE[c.dtype]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None] * len(cases)
    for _ in range(10):
        for i, c in enumerate(cases):
            got[i] = run_policy(c, ws=ws[i], stream=streams[i], **of(c))
    torch.cuda.synchronize()
    for i in range(len(cases)):
        assert L.lossk_device_status(ws[i]) == 580
        same(want[i], got[i])


@pytest.mark.parametrize("n,V,dtype,kw", [(20000, 16, "bf16", dict(seqs=7, masked=0.4)), (9000, 3, "f32", dict(masked=0.5)),
                                          (3, 300001, "f32", {}), (2, 500003, "f16", dict(seqs=2)),
                                          (300, 40, "f16", dict(seqs=200, empty=True))])
def test_many_rows_and_wide_ones(n, V, dtype, kw):
    c = Case(n, V, dtype, **kw)
    check_policy(c, run_policy(c, kl=0.1), kl=0.1)
    if c.first is not None:
        c.seq_adv = torch.randn(len(c.first) - 1, device="cuda", generator=gen(3))
        flags = L.SEQ_RATIO | L.SEQ_MEAN | L.SEQ_ADVANTAGES
        check_policy(c, run_policy(c, flags, low=0.013, high=0.017), flags, low=0.013, high=0.017)


def test_more_than_2_to_31_logits():
    """Rows past the 2^31st element: the last ones checked alone."""
    n, V = 14200, 151936
    logits = torch.empty(n, V, device="cuda", dtype=torch.bfloat16)
    g = gen(4)
    for i in range(0, n, 1000):
        logits[i:i + 1000] = torch.randn(min(1000, n - i), V, device="cuda", generator=g) * 2.0
    y = torch.randint(0, V, (n,), device="cuda", generator=g)
    adv = torch.randn(n, device="cuda", generator=g)
    old = torch.full((n,), -13.0, device="cuda")
    grad = torch.empty_like(logits)
    out = L.lossk_policy_from_logits(logits, y, adv, old, clip_high=9.0, clip_low=1.0, flags=L.REDUCE_SUM, grad_logits=grad)
    first = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
    pref = L.lossk_preference_from_logits(logits, y, first, flags=L.LENGTH_MEAN, want_grad=False)
    for t in (0, 7000, n - 1):
        lp = torch.log_softmax(logits[t].double(), -1)
        assert abs(float(out["logp"][t] - lp[y[t]])) < 1e-5 and abs(float(pref["logp"][t] - lp[y[t]])) < 1e-5
        r = math.exp(float(lp[y[t]]) + 13.0)
        a = float(adv[t])
        coef = a * r if (a <= 0 or r <= 10.0) else 0.0
        want = coef * torch.exp(lp)
        want[y[t]] -= coef
        assert torch.allclose(grad[t].double(), want, rtol=2.0 ** -8, atol=1e-4 * abs(coef) + 1e-12)
    # the gradient by pairs, of the last rows, on the same logits
    first = torch.tensor([0, 1, n], dtype=torch.int32, device="cuda")
    mask = torch.zeros(n, dtype=torch.uint8, device="cuda")
    mask[0] = mask[n - 1] = 1
    pref = L.lossk_preference_from_logits(logits, y, first, loss_mask=mask, beta=1.0, grad_logits=grad)
    lp = [torch.log_softmax(logits[t].double(), -1) for t in (0, n - 1)]
    u = float(lp[0][y[0]] - lp[1][y[n - 1]])
    for t, l, s in ((0, lp[0], 1.0), (n - 1, lp[1], -1.0)):
        coef = s / (1.0 + math.exp(u))
        want = coef * torch.exp(l)
        want[y[t]] -= coef
        assert torch.allclose(grad[t].double(), want, rtol=2.0 ** -8, atol=1e-4 * abs(coef) + 1e-12)
    assert not grad[1:n - 1:500].any()


def test_differences():
    """The gradient against differences of the total (fp32 logits, both losses)."""
    c = Case(n=12, V=50, dtype="f32", seqs=4, std=1.0)
    for run, kw in ((run_policy, dict(kl=0.3, flags=L.SEQ_RATIO, low=0.9, high=9.0)), (run_preference, dict(beta=0.4))):
        out = run(c, **kw)
        keep, g = c.logits.clone(), out["grad_logits"].double()
        rng = gen(6)
        for _ in range(6):
            v = torch.randn(c.n, c.V, device="cuda", generator=rng)
            step = 1e-2
            total = []
            for s in (step, -step):
                c.logits.copy_(keep + s * v)
                total.append(float(run(c, want_grad=False, **kw)["scalars"][0]))
            c.logits.copy_(keep)
            slope = (total[0] - total[1]) / (2 * step)
            want = float((g * v.double()).sum())
            # second order left out of a central difference: step^2 / 6 times a third derivative below 10 |v|^3
            assert abs(slope - want) < 2e-3 + 1e-2 * abs(want), (slope, want)
