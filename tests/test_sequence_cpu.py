"""The policy and preference losses on the CPU: refusals that come before any device work, the binding's checks, and the
64-bit reference's own checks (closed forms, differences)."""
import ctypes
import math
import types

import pytest
import torch

import output_projection_cross_gb300 as L
import seq_ref as R
from output_projection_cross_gb300 import sequence

P = 4096       # a 16-byte-aligned address that no call below gets to follow
BIG = 1 << 40


def policy_head(n=64, d=64, V=1000, n_seq=0, dtype=1, H=P, hl=BIG, W=P, wl=BIG, y=P, yl=BIG, mask=None, first=None, fl=0,
                adv=P, al=BIG, old=P, ol=BIG, ref=P, rl=BIG, low=0.2, high=0.2, kl=0.1, T=1.0, gs=1.0, flags=0, scal=P,
                per=None, lp=None, gd=0, dH=P, dW=P, ws=P, wsb=BIG):
    return L.lib.lossk_policy_fwd_bwd(n, d, V, n_seq, dtype, H, hl, W, wl, y, yl, mask, first, fl, adv, al, old, ol, ref, rl,
                                      low, high, kl, T, gs, flags, scal, per, lp, gd, dH, dW, ws, wsb, None)


def policy_logits(n=64, V=1000, n_seq=0, dtype=1, X=P, xl=BIG, y=P, yl=BIG, mask=None, first=None, fl=0, adv=P, al=BIG,
                  old=P, ol=BIG, ref=P, rl=BIG, low=0.2, high=0.2, kl=0.1, T=1.0, gs=1.0, flags=0, scal=P, per=None,
                  lp=None, g=P, gl=BIG, ws=P, wsb=BIG):
    return L.lib.lossk_policy_from_logits(n, V, n_seq, dtype, X, xl, y, yl, mask, first, fl, adv, al, old, ol, ref, rl, low,
                                          high, kl, T, gs, flags, scal, per, lp, g, gl, ws, wsb, None)


def pref_head(n=64, d=64, V=1000, pairs=2, dtype=1, H=P, hl=BIG, W=P, wl=BIG, y=P, yl=BIG, mask=None, first=P, fl=BIG,
              ref=P, rl=BIG, obj=0, beta=0.1, margin=0.0, smooth=0.0, nll=0.0, gs=1.0, flags=0, scal=P, gd=0, dH=P, dW=P,
              ws=P, wsb=BIG):
    return L.lib.lossk_preference_fwd_bwd(n, d, V, pairs, dtype, H, hl, W, wl, y, yl, mask, first, fl, ref, rl, obj, beta,
                                          margin, smooth, nll, gs, flags, scal, None, None, None, gd, dH, dW, ws, wsb, None)


def pref_logits(n=64, V=1000, pairs=2, dtype=1, X=P, xl=BIG, y=P, yl=BIG, mask=None, first=P, fl=BIG, ref=P, rl=BIG, obj=0,
                beta=0.1, margin=0.0, smooth=0.0, nll=0.0, gs=1.0, flags=0, scal=P, g=P, gl=BIG, ws=P, wsb=BIG):
    return L.lib.lossk_preference_from_logits(n, V, pairs, dtype, X, xl, y, yl, mask, first, fl, ref, rl, obj, beta, margin,
                                              smooth, nll, gs, flags, scal, None, None, None, g, gl, ws, wsb, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("f", [policy_head, policy_logits, pref_head, pref_logits])
def test_refusals_all_share(f):
    head, pref = f in (policy_head, pref_head), f in (pref_head, pref_logits)
    assert f(n=0) == f(V=0) == 581
    assert f(n=(1 << 24) + 1) == f(V=(1 << 24) + 1) == 583
    if head:
        assert f(d=0) == 581 and f(n=1 << 16, d=1 << 15, V=(1 << 15) + 8) == 584
        for bad in (dict(H=None), dict(W=None), dict(hl=64 * 64 - 1), dict(wl=64000 - 1), dict(gd=2), dict(gd=7)):
            assert f(**bad) == 582, bad
        for bad in (dict(H=P + 8), dict(W=P + 2), dict(dH=P + 4), dict(dW=P + 8), dict(d=60)):
            assert f(**bad) == 591, bad
        assert f(gd=1, flags=1) == f(gd=1, flags=1, dH=None) == f(gd=1, flags=1, dW=None) == 592
    else:
        for bad in (dict(X=None), dict(xl=63999), dict(gl=63999)):
            assert f(**bad) == 582, bad
        for bad in (dict(X=P + 8), dict(g=P + 4)):
            assert f(**bad) == 591, bad
    for bad in (dict(dtype=3), dict(dtype=-1), dict(y=None), dict(yl=63), dict(scal=None), dict(ws=None), dict(wsb=255),
                dict(rl=63), dict(first=P, fl=2, **({} if pref else dict(n_seq=2)))):
        assert f(**bad) == 582, bad
    assert f(ws=P + 128) == 591
    for bad in (NAN, INF):
        assert f(gs=bad) == 585
    assert f(flags=64) == f(flags=1 << 31) == 592


@pytest.mark.parametrize("f", [policy_head, policy_logits])
def test_refusals_of_the_policy_loss(f):
    assert f(n_seq=-1, first=P, fl=BIG) == 581
    assert f(n_seq=(1 << 25) + 1, first=P, fl=BIG) == 583
    for bad in (dict(first=P, fl=9), dict(n_seq=3), dict(adv=None), dict(al=63), dict(ol=63), dict(ref=None),
                dict(flags=4), dict(flags=8), dict(flags=16), dict(n_seq=3, first=P, fl=4, flags=16, al=2)):
        assert f(**bad) == 582, bad
    for bad in (dict(low=-0.1), dict(low=1.1), dict(high=-0.1), dict(kl=-1.0), dict(T=0.0), dict(T=-1.0), dict(T=NAN),
                dict(low=NAN), dict(high=INF), dict(kl=INF), dict(T=INF), dict(T=1e-31), dict(T=1e31), dict(high=1e39), dict(kl=1e39), dict(gs=1e39)):
        assert f(**bad) == 585, bad
    assert f(flags=32) == 592


@pytest.mark.parametrize("f", [pref_head, pref_logits])
def test_refusals_of_the_preference_loss(f):
    assert f(pairs=0) == f(pairs=-3) == 581 and f(pairs=(1 << 24) + 1) == 583
    assert f(first=None) == f(fl=4) == 582
    for bad in (dict(beta=0.0), dict(beta=-1.0), dict(beta=NAN), dict(margin=INF), dict(smooth=-0.1), dict(smooth=1.1),
                dict(nll=-1.0), dict(nll=NAN), dict(beta=1e-31), dict(beta=1e39), dict(margin=1e39), dict(nll=1e39), dict(obj=1, margin=0.1), dict(obj=2, smooth=0.1)):
        assert f(**bad) == 585, bad
    assert f(obj=3) == f(obj=-1) == 588
    for flag in (4, 8, 16):
        assert f(flags=flag) == 592


def test_workspace_sizes():
    size = L.lossk_sequence_workspace_bytes
    for kind in (0, 1):
        for dtype in (0, 1, 2):
            nb = size(kind, 300, 64, 1000, 6, dtype)
            assert nb > 256 and nb % 256 == 0 and size(kind, 300, 64, 1000, 0, dtype) <= nb
    assert size(2, 300, 64, 1000, 0, 1) == size(0, 0, 64, 1000, 0, 1) == size(0, 300, 64, 1000, -1, 1) == -1
    assert size(0, 300, 0, 1000, 0, 1) == -1 and size(1, 300, 0, 1000, 0, 1) > 0 and size(1, 300, 0, 1000, 0, 5) == -1
    with pytest.raises(L.LosskError):
        L.sequence_workspace(0, 0, 64, 1000, 0, 1)


def test_kernel_names():
    names = [L.lossk_kernel_name(i) for i in range(L.lossk.N_KERNELS)]
    assert "unknown_kernel" not in names and len(set(names)) == len(names)
    assert L.lossk_kernel_name(L.lossk.N_KERNELS) == "unknown_kernel"


def test_module_and_ctypes_agree():
    """The CPython module takes the arguments in the same places as ctypes."""
    from output_projection_cross_gb300 import decode
    if isinstance(decode._calls, decode._NotBuilt):
        pytest.skip("without Python's headers there is no module")
    kinds = {"c_void_p": None, "c_double": 0.0}
    for name in ("lossk_policy_fwd_bwd", "lossk_policy_from_logits", "lossk_preference_fwd_bwd",
                 "lossk_preference_from_logits"):
        f, g = getattr(decode._calls, name), getattr(L.lib, name)
        args = [kinds.get(t.__name__, 0) for t in g.argtypes]
        assert f(*args) == g(*args) != 580
        for i, a in enumerate(args):
            if a == 0 and not isinstance(a, float):
                args[i] = 1
                assert f(*args) == g(*args) != 580, (name, i)
        with pytest.raises(TypeError):
            f(*args[:-1])


class Reached(Exception):
    pass


class OnGpu:
    """A CPU tensor that says it is on a GPU."""

    def __init__(self, t, index=0):
        self.t, self.index, self.is_cuda = t, index, index >= 0

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def library(monkeypatch):
    got = {}

    def reached(*args):
        got["args"] = args
        raise Reached
    names = ("lossk_policy_fwd_bwd", "lossk_policy_from_logits", "lossk_preference_fwd_bwd", "lossk_preference_from_logits")
    monkeypatch.setattr(sequence, "_lib", types.SimpleNamespace(**{n: reached for n in names}))
    monkeypatch.setattr(sequence, "_stream_of", lambda stream, *t: 0)
    return got


def tensors(name):
    n, d, V = 6, 8, 5
    t = dict(targets=torch.zeros(n, dtype=torch.int64), ws=torch.zeros(256, dtype=torch.uint8),
             loss_mask=torch.ones(n, dtype=torch.uint8), ref_logp=torch.zeros(n), scalars_out=torch.zeros(4),
             logp_out=torch.zeros(n))
    t.update(dict(hidden=torch.zeros(n, d), weight=torch.zeros(V, d), d_hidden=torch.zeros(n, d),
                  d_weight=torch.zeros(V, d)) if name.endswith("bwd") else
             dict(logits=torch.zeros(n, V), grad_logits=torch.zeros(n, V)))
    if "policy" in name:
        t.update(advantages=torch.zeros(n), old_logp=torch.zeros(n), per_token_out=torch.zeros(n),
                 first=torch.zeros(3, dtype=torch.int32))
    else:
        t.update(first=torch.zeros(5, dtype=torch.int32), per_pair_out=torch.zeros(2), log_ratio_out=torch.zeros(4))
    return t


NAMES = ["lossk_policy_fwd_bwd", "lossk_policy_from_logits", "lossk_preference_fwd_bwd", "lossk_preference_from_logits"]


@pytest.mark.parametrize("name", NAMES)
def test_binding_checks_types_sizes_and_layout(name, library):
    f, good = getattr(L, name), tensors(name)
    with pytest.raises(Reached):
        f(**good)
    for k, t in good.items():
        if k in ("hidden", "weight", "logits"):
            continue
        wrong = t.to(torch.float64) if t.dtype != torch.float64 else t.float()
        with pytest.raises(TypeError):
            f(**{**good, k: wrong})
    for k in ("targets", "loss_mask", "scalars_out", "logp_out"):
        with pytest.raises(ValueError):
            f(**{**good, k: good[k][:-1]})
    for k in ("hidden", "weight", "logits", "grad_logits", "d_hidden", "d_weight"):
        if k in good:
            t = good[k]
            with pytest.raises(ValueError):
                f(**{**good, k: torch.zeros(t.shape[1], t.shape[0], dtype=t.dtype).t()})
            with pytest.raises((ValueError, Reached)) as e:
                f(**{**good, k: t[:-1]})
            assert k in ("logits", "weight") or e.type is ValueError or k == "hidden"
    if "preference" in name:
        with pytest.raises(ValueError):
            f(**{**good, "first": torch.zeros(4, dtype=torch.int32)})
        with pytest.raises(KeyError):
            f(**good, objective="cosine")


@pytest.mark.parametrize("name", [n for n in NAMES if n.endswith("bwd")])
def test_binding_gradient_types(name, library):
    f, good = getattr(L, name), tensors(name)
    for k in ("hidden", "weight"):
        good[k] = good[k].to(torch.bfloat16)
    for dtype, want in ((torch.float32, 0), (torch.bfloat16, 1)):
        given = {**good, "d_hidden": good["d_hidden"].to(dtype), "d_weight": good["d_weight"].to(dtype)}
        with pytest.raises(Reached):
            f(**given)
        assert library["args"][-6] == want
        with pytest.raises(TypeError):
            f(**given, grad_dtype=torch.float16)
    with pytest.raises(TypeError):
        f(**{**good, "d_weight": good["d_weight"].to(torch.bfloat16)})


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_another_gpu(name, monkeypatch):
    from output_projection_cross_gb300 import decode
    if isinstance(decode._calls, decode._NotBuilt):
        pytest.skip("without Python's headers there is no module")

    def reached(*args):
        raise Reached
    monkeypatch.setattr(sequence, "_lib", types.SimpleNamespace(**{n: reached for n in NAMES}))
    monkeypatch.setattr(decode, "_current_device", lambda: 0)
    monkeypatch.setattr(decode, "_raw_stream", lambda i: 0)
    f, good = getattr(L, name), {k: OnGpu(t) for k, t in tensors(name).items()}
    with pytest.raises(Reached):
        f(**good)
    for k in good:
        for index in (1, -1):
            with pytest.raises(ValueError):
                f(**{**good, k: OnGpu(good[k].t, index)})


def test_reference_policy_closed_forms():
    lp = torch.tensor([-1.0, -2.0, -3.0, -4.0], dtype=torch.float64)
    on = torch.tensor([True, True, True, False])
    # ratios 1.5 (clipped for A > 0), 1 and 0.5 (clipped for A < 0)
    old = lp - torch.tensor([1.5, 1.0, 0.5, 1.0], dtype=torch.float64).log()
    adv = torch.tensor([2.0, -1.0, -4.0, 9.0], dtype=torch.float64)
    r = R.policy(lp, on, None, adv, old, None)
    assert torch.allclose(r["per_token"], torch.tensor([-2.4, 1.0, 3.2, 0.0], dtype=torch.float64))
    assert torch.allclose(r["slope"], torch.tensor([0.0, 1.0 / 3, 0.0, 0.0], dtype=torch.float64))
    assert torch.allclose(r["scalars"], torch.tensor([1.8 / 3, 1.8 / 3, 0.0, 2.0 / 3], dtype=torch.float64))
    # the KL term of a reference log 2 above: 2 - log 2 - 1
    r = R.policy(lp, on, None, torch.zeros(4).double(), None, lp + math.log(2.0), kl=1.0)
    assert torch.allclose(r["per_token"][:3], torch.full((3,), 1.0 - math.log(2.0), dtype=torch.float64))
    assert torch.allclose(r["slope"][:3], torch.full((3,), -1.0 / 3, dtype=torch.float64))


@pytest.mark.parametrize("flags", [(False, False), (True, False), (False, True), (True, True)])
def test_reference_slopes_are_differences(flags):
    g = torch.Generator().manual_seed(1)
    lp = -torch.rand(12, generator=g, dtype=torch.float64) * 4
    first, on = torch.tensor([0, 5, 5, 11]), torch.rand(12, generator=g) > 0.2
    on[11:] = False
    old, ref = lp - 0.05 * torch.randn(12, generator=g, dtype=torch.float64), lp + torch.randn(12, generator=g).double()
    adv = torch.randn(12, generator=g, dtype=torch.float64)
    f = lambda x: R.policy(x, on, first, adv, old, ref, 0.3, 0.3, 0.1, seq_ratio=flags[0], seq_mean=flags[1])  # noqa: E731
    base = f(lp)
    for i in range(12):
        e = torch.zeros(12, dtype=torch.float64)
        e[i] = 1e-6
        d = (f(lp + e)["scalars"][0] - f(lp - e)["scalars"][0]) / 2e-6
        assert abs(float(d - base["slope"][i])) < 1e-8


@pytest.mark.parametrize("opts", [dict(), dict(margin=0.3, smoothing=0.1), dict(objective="hinge"),
                                  dict(objective="squared", beta=0.7), dict(nll=0.5, length_mean=True), dict(summed=True)])
def test_reference_preference_slopes_are_differences(opts):
    g = torch.Generator().manual_seed(2)
    lp = -torch.rand(14, generator=g, dtype=torch.float64) * 4
    first, on = torch.tensor([0, 4, 7, 10, 13]), torch.ones(14, dtype=torch.bool)
    on[[1, 13]] = False
    ref = lp + 0.3 * torch.randn(14, generator=g, dtype=torch.float64)
    f = lambda x: R.preference(x, on, first, ref, **opts)  # noqa: E731
    base = f(lp)
    for i in range(14):
        e = torch.zeros(14, dtype=torch.float64)
        e[i] = 1e-6
        d = (f(lp + e)["scalars"][0] - f(lp - e)["scalars"][0]) / 2e-6
        assert abs(float(d - base["slope"][i])) < 1e-7
    assert float(base["slope"][1]) == float(base["slope"][13]) == 0.0


def test_reference_preference_closed_form():
    # equal log ratios: log 2, half of beta each way
    lp = torch.tensor([-1.0, -2.0], dtype=torch.float64)
    r = R.preference(lp, torch.ones(2, dtype=torch.bool), torch.tensor([0, 1, 2]), lp.clone(), beta=0.4)
    assert abs(float(r["scalars"][0]) - math.log(2.0)) < 1e-15 and float(r["scalars"][3]) == 0.0
    assert torch.allclose(r["slope"], torch.tensor([-0.2, 0.2], dtype=torch.float64))


def test_signatures_match_the_header():
    """As many arguments in ctypes' table as in lossk.h, pointers where there are pointers."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "lossk.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    kind = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "uint32_t": ctypes.c_uint32, "double": ctypes.c_double,
            "lossk_stream_t": ctypes.c_void_p}
    for name in (*NAMES, "lossk_sequence_workspace_bytes"):
        args = re.search(r"\b%s\s*\(([^)]*)\)" % name, src).group(1).split(",")
        want = [ctypes.c_void_p if "*" in a else kind[a.split()[0]] for a in args]
        assert getattr(L.lib, name).argtypes == want, name
