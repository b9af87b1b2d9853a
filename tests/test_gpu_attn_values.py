"""Attention over a paged cache on values that are hard for it: one token that outweighs a long tail,
scores that rise and fall from tile to tile.

Many sequences list the same pages, so that a warp's run is many tiles of one sequence; one sequence is
the reference for all.  Bounds as in test_gpu_attn.py: half a step of the output's type, and of the
weighted mean of |v| what the fp32 sums and exponents (of up to 40 in log2 units) carry.  fp16 outputs
below 2^-14 are off by up to 2^-25, half their step there, and weights in one tile with a token that
outweighs them by 2^d by up to 2^-32 of it each, 16 of them: 2^-24 covers both for |v| up to 8.
"""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PAGE, KV, HD = 16, 8, 64


@pytest.fixture(scope="module")
def L():
    from conftest import build_lib
    build_lib()
    import output_projection_cross_gb300 as L
    assert torch.cuda.is_available()
    return L


def check(L, scores, v, dtype, group, share=1, seqs=48):
    """Every token's score is scores[j]; v [tokens].  All heads and sequences are alike."""
    n, dt = len(scores), DTYPES[dtype]
    k = torch.zeros((-(-n // PAGE), PAGE, KV, HD), device="cuda", dtype=dt)
    vals = torch.zeros_like(k)
    # a score as the sum of parts that the type holds (scores are multiples of 2^-4, below 2^7)
    flat = torch.zeros((k.shape[0] * PAGE, HD), device="cuda", dtype=dt)
    flat[:n, 0] = torch.from_numpy(np.floor(scores)).cuda().to(dt)
    flat[:n, 1] = torch.from_numpy(scores - np.floor(scores)).cuda().to(dt)
    k[:] = flat.view(k.shape[0], PAGE, 1, HD)
    flat = torch.zeros((k.shape[0] * PAGE,), device="cuda", dtype=dt)
    flat[:n] = torch.from_numpy(v).cuda().to(dt)
    vals[:] = flat.view(k.shape[0], PAGE, 1, 1)
    hq = KV * group
    q = torch.zeros((seqs, hq, HD), device="cuda", dtype=dt)
    q[:, :, :2] = 1.0
    table = torch.arange(k.shape[0], dtype=torch.int32, device="cuda").expand(seqs, -1).contiguous()
    ws = L.decode_workspace(L.KIND_PAGED_ATTN, seqs, hq, KV, HD)
    lse = torch.empty((seqs, hq), device="cuda")
    out = L.lossk_paged_attn(q, k, vals, table, torch.full((seqs,), n, dtype=torch.int32, device="cuda"), scale=1.0,
                             share=share, lse_out=lse, ws=ws)
    assert L.lossk_device_status(ws) == 580
    one = (x[:, :, :1].double().cpu().numpy() for x in (k, vals))
    kd, vd = one
    args = table[:1].cpu().numpy(), [n], PAGE, 1.0
    r, rl = ref.attend(q[:1, :1].double().cpu().numpy(), kd, vd, *args)
    mean, _ = ref.attend(q[:1, :1].double().cpu().numpy(), kd, np.abs(vd), *args)
    got = out.double().cpu().numpy()
    eps, x_err = torch.finfo(dt).eps, 2.0 ** -24 * (40 * (HD / 8 + 8) + 64)
    bound = eps / 2 * np.abs(r) + x_err * mean + (2.0 ** -24 if dtype == "f16" else 0)
    assert np.isfinite(got).all()
    assert (np.abs(got - r) <= bound).all(), (np.abs(got - r).max(), r.flat[0], bound.flat[0])
    assert (np.abs(lse.double().cpu().numpy() - rl) <= 2.0 ** -24 * np.abs(rl) + x_err).all()


def tail(n, seed=0):
    """Scores of a tail about 0 and its values, about 1."""
    rng = np.random.default_rng(seed)
    return np.round(rng.standard_normal(n) * 8) / 16, rng.uniform(0.5, 1.5, n)


@pytest.mark.parametrize("at", [0, 7, 2000, 4095])
@pytest.mark.parametrize("d", [5, 12, 14, 16, 18, 20, 60])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_one_token_of_value_zero_over_a_long_tail(L, dtype, d, at):
    s, v = tail(4096)
    s[at], v[at] = d, 0.0
    check(L, s, v, dtype, 1)


@pytest.mark.parametrize("group,share", [(1, 4), (20, 1), (5, 4), (40, 1), (8, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_of_many_query_rows(L, dtype, group, share):
    s, v = tail(4090, 1)
    s[3], v[3] = 18, 0.0
    check(L, s, v, dtype, group, share)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_scores_that_rise_and_fall(L, dtype):
    s, v = tail(4096, 2)
    for period, step in ((16, 16.0), (48, 20.0), (160, 11.0)):
        check(L, s + step * (np.arange(4096) // period % 2), v * np.where(np.arange(4096) // period % 2, 0.0, 1.0),
              dtype, 1)
    check(L, s + np.floor(np.arange(4096) / 64), v, dtype, 1)
    check(L, s + np.floor(np.arange(4095, -1, -1) / 64), v, dtype, 1)


@pytest.mark.parametrize("d", [16, 30, 45, 100])
def test_large_values_under_a_small_weight(L, d):
    """fp16's largest values times weights that are taken up to 2^75 for them: no overflow on the way.
    (The heavy token's tile has no values: beside it they would be off by 2^-32 of 40000 each.)"""
    s, v = tail(4096, 3)
    v *= 40000.0
    s[0], v[:16] = d, 0.0
    check(L, s, np.floor(v), "f16", 1)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,kv,hd,share,lens", [
    (4, 2, 64, 1, [1, 37, 300, 16]), (40, 2, 128, 1, [200, 5, 90]), (80, 1, 72, 1, [130, 33]),
    (8, 2, 96, 4, [150, 150, 170, 149]), (3, 3, 200, 1, [64, 9000]), (8, 1, 256, 2, [70, 75])])
def test_infinite_values(L, dtype, hq, kv, hd, share, lens):
    """A value of infinity under a positive weight is infinity, under both signs of it no number; what the
    other columns hold is what it was."""
    rng = np.random.default_rng([hq, hd])
    S, dt = len(lens), DTYPES[dtype]
    used = [-(-n // PAGE) for n in lens]
    table = np.full((S, max(used)), -1, np.int32)
    table[:] = np.arange(max(used))
    if share == 1:
        for s in range(S):
            table[s] += sum(used[:s])
    n_pages = int(table.max()) + 1
    k = torch.from_numpy(rng.standard_normal((n_pages, PAGE, kv, hd))).cuda().to(dt)
    v = torch.from_numpy(rng.standard_normal((n_pages, PAGE, kv, hd))).cuda().to(dt)
    q = torch.from_numpy(rng.standard_normal((S, hq, hd))).cuda().to(dt)
    t, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    inf = float("inf")
    for page in range(0, n_pages, 3):
        v[page, 0, :, 0:4] = inf
        v[page, 3, :, 4:6] = -inf
        v[page, 0, :, 6], v[page, 9, :, 6] = inf, -inf
        v[page, 2, 0, 7] = float("nan")
        v[page, 15, :, hd - 1] = inf
    for window in (0, 20):
        ws = L.decode_workspace(L.KIND_PAGED_ATTN, S, hq, kv, hd)
        lse = torch.empty((S, hq), device="cuda")
        out = L.lossk_paged_attn(q, k, v, t, n, share=share, window=window, lse_out=lse, ws=ws)
        assert L.lossk_device_status(ws) == 580
        with np.errstate(invalid="ignore"):
            args = table, lens, PAGE, hd ** -0.5, window
            r, rl = ref.attend(*(x.double().cpu().numpy() for x in (q, k, v)), *args)
            mean, _ = ref.attend(*(x.double().cpu().numpy() for x in (q, k, v.abs())), *args)
        assert np.isposinf(r).any() and np.isfinite(r).any() and (window or np.isneginf(r).any() and np.isnan(r).any())
        got = out.double().cpu().numpy()
        fin = np.isfinite(r)
        np.testing.assert_array_equal(got[~fin], r[~fin])
        x_err = 2.0 ** -24 * (40 * (hd / 8 + 8) + 64)
        bound = torch.finfo(dt).eps / 2 * np.abs(r[fin]) + x_err * mean[fin] + (2.0 ** -24 if dtype == "f16" else 0)
        assert (np.abs(got[fin] - r[fin]) <= bound).all()
        assert (np.abs(lse.double().cpu().numpy() - rl) <= 2.0 ** -24 * np.abs(rl) + x_err).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_infinite_keys(L, dtype):
    """A key that makes a score -infinity takes its token out."""
    rng = np.random.default_rng(5)
    dt = DTYPES[dtype]
    k, v = (torch.from_numpy(rng.standard_normal((5, PAGE, 2, 64))).cuda().to(dt) for _ in range(2))
    q = torch.from_numpy(rng.uniform(0.5, 1.5, (1, 4, 64))).cuda().to(dt)
    table = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    k[1, 4, :, 3] = -float("inf")
    k[3, :, :, 9] = -float("inf")
    out = L.lossk_paged_attn(q, k, v, table, torch.tensor([75], dtype=torch.int32, device="cuda"))
    r, _ = ref.attend(*(x.double().cpu().numpy() for x in (q, k, v)), table.cpu().numpy(), [75], PAGE, 0.125)
    mean, _ = ref.attend(*(x.double().cpu().numpy() for x in (q, k, v.abs())), table.cpu().numpy(), [75], PAGE, 0.125)
    x_err = 2.0 ** -24 * (40 * (64 / 8 + 8) + 64)
    bound = torch.finfo(dt).eps / 2 * np.abs(r) + x_err * mean + (2.0 ** -24 if dtype == "f16" else 0)
    assert (np.abs(out.double().cpu().numpy() - r) <= bound).all()
