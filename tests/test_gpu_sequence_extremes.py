"""The policy and preference losses at the ends of their arguments: the smallest head sizes in each type, more tokens or
sequences than a kernel numbers in one round, coefficients of zero and far below one, calls from two threads, and the
losses one after another as a training run has them."""
import threading

import pytest
import torch

import output_projection_cross_gb300 as L
import seq_ref as R
from test_gpu_sequence import CODE, DT, HALF, Case, check_grads, check_policy, check_preference, close, run_policy, run_preference
from test_gpu_sequence_edges import of, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,V,d,dtype", [(1, 1, 8, "f16"), (1, 1, 8, "bf16"), (1, 1, 1, "f32"), (1, 2, 3, "f32"), (2, 300, 8, "f16"),
                                         (1, 5000, 64, "f16"), (1, 5000, 64, "bf16"), (1, 5000, 65, "f32"),
                                         (20000, 40, 8, "bf16"), (9000, 33, 16, "f16"), (9000, 17, 5, "f32"),
                                         (70, 500, 4104, "bf16"), (70, 500, 4104, "f16"), (40, 300, 2049, "f32")])
def test_head_sizes(n, V, d, dtype):
    c = Case(n, V, dtype, d=d, masked=0.2 if n > 2 else 0.0, seqs=4 if n >= 8 else 0)
    check_policy(c, run_policy(c, kl=0.1, **of(c)), kl=0.1)
    if c.first is not None:
        check_preference(c, run_preference(c, **of(c)))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("low", [3.0, 12.0, 60.0, 150.0])
def test_every_logit_is_low(dtype, low):
    """Vocabularies that end inside a tile, every logit far below 0: what lies past the end stays out."""
    for V in (300, 1001):
        c = Case(n=40, V=V, d=64, dtype=dtype, std=0.5)
        c.hidden[:, 0], c.weight[:, 0] = -4.0, low / 4.0
        c.x = c.hidden.double() @ c.weight.double().t()
        c.fill(torch.Generator(device="cuda").manual_seed(3))
        assert float(c.x.logsumexp(1).max()) < 0 or low < 10
        check_policy(c, run_policy(c, kl=0.1, **of(c)), kl=0.1)
        got = L.lossk_ce_fwd_bwd(c.hidden, c.weight, c.targets, chunk=64)
        g, a = R.grad_logits(c.x, c.targets, c.on, torch.full((c.n,), -1.0 / c.n, device="cuda", dtype=torch.float64))
        # A tile's entries p / n and (p - 1) / n are rounded to 16 bits (fp16: to 2^-24 of 1 / n at the least) and moved by
        # the error of lse; what a gradient sums them with does not cancel: a column of 37.5 times the entries' sum, 0,
        # is off by up to 75 half steps.
        own = torch.softmax(c.x, -1) / c.n
        own[torch.arange(c.n), c.targets] += 1.0 / c.n
        err = ((HALF[dtype] if dtype != "f32" else 0.0) + 8 * c.lp_tol() + 2.0 ** -20) * own + 2.0 ** -24 / c.n
        h, w = c.hidden.double(), c.weight.double()
        for k, want, tol in (("d_hidden", g @ w, err @ w.abs()), ("d_weight", g.t() @ h, err.t() @ h.abs())):
            close(got[k], want, tol + 2.0 ** -20 * want.abs(), k)


@pytest.mark.parametrize("kw", [dict(n=40, V=900, dtype="bf16"), dict(n=40, V=300, d=64, dtype="bf16"),
                                dict(n=40, V=300, d=20, dtype="f32")], ids=str)
def test_more_sequences_than_tokens(kw):
    c = Case(seqs=4, **kw)
    want = run_policy(c, L.SEQ_RATIO | L.SEQ_MEAN, **of(c))
    # the same sequences among 5000 empty ones
    f = c.first.cpu()
    at = torch.zeros(5001, dtype=torch.int32)
    at[:1000], at[1000:2500], at[2500:4000], at[4000:4999], at[4999:] = f[0], f[1], f[2], f[3], f[4]
    c.first = at.to("cuda")
    got = run_policy(c, L.SEQ_RATIO | L.SEQ_MEAN, **of(c))
    for k in ("per_token", "logp", "d_hidden", "grad_logits"):
        if want.get(k) is not None:
            assert torch.equal(want[k], got[k]), k
    close(got["scalars"], want["scalars"].double(), 2.0 ** -22 * (1.0 + want["scalars"].double().abs()), "scalars")


@pytest.mark.parametrize("kw", [dict(n=70, V=900, d=136, dtype="f16"), dict(n=70, V=900, d=136, dtype="bf16"),
                                dict(n=70, V=900, d=72, dtype="f32"), dict(n=70, V=9000, dtype="f16")], ids=str)
@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e20])
def test_scales_of_the_gradient(kw, scale):
    c = Case(**kw)
    kwargs = dict(grad_dtype=torch.float32) if c.d else {}
    out = run_policy(c, kl=0.1, grad_scale=scale, **kwargs)
    grads = [out[k] for k in ("d_hidden", "d_weight", "grad_logits") if out.get(k) is not None]
    if scale == 0.0:
        assert not any(g.any() for g in grads)
    elif c.d:
        r = R.policy(c.lp, c.on, c.first, c.adv, c.old, c.ref, kl=0.1)
        check_grads(c, out, r, scale=scale, grad="float")
    elif scale > 1.0:
        assert all(torch.isinf(g).any() for g in grads)    # beyond fp16


def test_two_threads():
    """Calls of both losses from two threads, on streams of their own."""
    cases = [Case(n=150, V=3000, d=136, dtype="bf16", seqs=4, seed=1), Case(n=150, V=3000, d=136, dtype="f16", seqs=4, seed=2)]
    want = [(run_policy(c, **of(c)), run_preference(c, **of(c))) for c in cases]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            c, s = cases[i], torch.cuda.Stream()
            ws = L.sequence_workspace(0, c.n, c.d, c.V, 4, CODE[c.dtype])
            torch.cuda.synchronize()
            for _ in range(20):
                a, b = run_policy(c, ws=ws, stream=s, **of(c)), run_preference(c, ws=ws, stream=s, **of(c))
            s.synchronize()
            same(want[i][0], a)
            same(want[i][1], b)
            with torch.cuda.stream(s):
                assert L.lossk_device_status(ws) == 580
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_a_run_of_them(dtype):
    """Label loss, log-probabilities before and of a reference, policy steps, a preference step: one head, each step's
    gradient against the 64-bit definitions at the weights that it ran on."""
    c = Case(n=96, V=1200, d=64, dtype=dtype, seqs=4, masked=0.2)
    weight, T = c.weight.clone(), DT[dtype]
    given = lambda: dict(first=c.first, loss_mask=c.mask)  # noqa: E731
    ws = L.sequence_workspace(0, c.n, c.d, c.V, 4, CODE[dtype])
    zero = torch.zeros(c.n, device="cuda")
    forward = dict(want_d_hidden=False, want_d_weight=False, ws=ws)

    def step(grad, rate):
        size = grad.float().abs().max()
        c.weight = (c.weight.float() - rate * grad.float() / size).to(T)
        c.x = torch.where(c.on[:, None], c.hidden.double(), 0.0) @ c.weight.double().t()
        c.lp = R.logprobs(c.x, c.targets, c.on)

    ref = L.lossk_policy_fwd_bwd(c.hidden, weight, c.targets, zero, **given(), **forward)["logp"]
    close(ref, c.lp, c.lp_tol() + 2.0 ** -24 * c.lp.abs(), "reference")
    h = torch.where(c.on[:, None], c.hidden, torch.zeros((), device="cuda", dtype=T))
    y = torch.where(c.on, c.targets, 0)
    label = L.lossk_ce_fwd_bwd(h, c.weight, y, loss_mask=c.on.to(torch.uint8), chunk=64)
    step(label["d_weight"], 0.01)
    c.ref = ref
    c.old = L.lossk_policy_fwd_bwd(c.hidden, c.weight, c.targets, zero, **given(), **forward)["logp"]
    for _ in range(2):
        # (a clamp that no ratio comes near: after a step they are not kept from its borders)
        out = run_policy(c, kl=0.05, low=0.9, high=9.0, ws=ws, **of(c))
        check_policy(c, out, kl=0.05, low=0.9, high=9.0)
        step(out["d_weight"], 0.002)
    out = run_preference(c, ws=ws, **of(c))
    check_preference(c, out)
    assert L.lossk_device_status(ws) == 580


@pytest.mark.parametrize("kw", [dict(n=37, V=901, d=72, dtype="bf16"), dict(n=37, V=901, d=72, dtype="f16"),
                                dict(n=37, V=901, d=19, dtype="f32"), dict(n=300, V=2000, d=264, dtype="bf16"),
                                dict(n=37, V=1001, dtype="bf16"), dict(n=37, V=9001, dtype="f16"), dict(n=5, V=40003, dtype="f32"),
                                dict(n=2, V=120001, dtype="bf16"), dict(n=2, V=500003, dtype="bf16")], ids=str)
@pytest.mark.parametrize("grad", ["same", "float"])
def test_nothing_is_written_beside_the_outputs(kw, grad):
    """Each output and the workspace in the middle of a larger buffer; the workspace but its header begins as 0xFF."""
    c = Case(seqs=4 if kw["n"] > 4 else 2, masked=0.2 if kw["n"] > 4 else 0.0, **kw)
    if not c.d and grad == "float":
        pytest.skip("grad_logits is of the logits' type")
    n, V, d, seqs = c.n, c.V, c.d, len(c.first) - 1
    kind = 0 if c.d else 1
    gt = torch.float32 if grad == "float" else DT[c.dtype]
    kept = []

    def inside(shape, dtype):
        size = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        whole = torch.full((4096 + size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        kept.append((whole, size))
        return whole[4096:4096 + size].view(dtype).view(shape)

    f32 = torch.float32
    ws = inside((L.lossk_sequence_workspace_bytes(kind, n, max(d, 1), V, seqs, CODE[c.dtype]),), torch.uint8)
    ws[256:] = 0xFF
    ws[:256] = 0
    outs = dict(scalars_out=inside((4,), f32), logp_out=inside((n,), f32), ws=ws)
    if c.d:
        outs.update(d_hidden=inside((n, d), gt), d_weight=inside((V, d), gt))
    else:
        outs.update(grad_logits=inside((n, V), gt))
    kwargs = dict(grad="float") if c.d and grad == "float" else {}
    check_policy(c, run_policy(c, kl=0.1, per_token_out=inside((n,), f32), **outs), kl=0.1, **kwargs)
    ws[256:] = 0xFF
    check_policy(c, run_policy(c, L.SEQ_RATIO, low=0.013, high=0.017, **outs), L.SEQ_RATIO, low=0.013, high=0.017, **kwargs)
    ws[256:] = 0xFF
    check_preference(c, run_preference(c, per_pair_out=inside((seqs // 2,), f32), log_ratio_out=inside((seqs,), f32), **outs),
                     **kwargs)
    for whole, size in kept:
        assert (whole[:4096] == 0xA5).all() and (whole[4096 + size:] == 0xA5).all()


def test_graphs_that_share_a_workspace():
    """Two graphs recorded with one workspace, replayed in turn on one stream."""
    a, b = Case(n=70, V=900, d=136, dtype="bf16", seqs=4, seed=1), Case(n=60, V=900, d=136, dtype="bf16", seqs=4, seed=2)
    want = run_policy(a, **of(a)), run_preference(b, **of(b))
    ws = L.sequence_workspace(0, 70, 136, 900, 4, CODE["bf16"])
    graphs, got, stream = [], [], torch.cuda.Stream()
    for run, c in ((run_policy, a), (run_preference, b)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            got.append(run(c, ws=ws, **of(c)))
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    same(want[0], got[0])
    same(want[1], got[1])
