"""Selection where logits over the temperature are large: 1e8 to 1e30, as an additive mask leaves whole rows.

Bounds: score and log-sum-exp round to float (2^-24 of the value); the log-sum-exp's own error is 3e-6 as for
small logits; products and sums of doubles of the size of logits / temperature are off by 4 half steps, 2^-51 of it.
"""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def L():
    from conftest import build_lib
    build_lib()
    import output_projection_cross_gb300 as L
    assert torch.cuda.is_available()
    return L


def check(L, x, n_out, temperature):
    rows, V = x.shape
    s = np.array([[-0.25, -3.5]], np.float32)
    assert rows == 2
    ws = L.decode_workspace(L.KIND_BEAM_SELECT, 1, 2, V, n_out)
    lse = torch.empty(2, device="cuda")
    o = L.lossk_beam_select(x, torch.from_numpy(s).cuda(), n_out, temperature=temperature, lse_out=lse, ws=ws)
    assert L.lossk_device_status(ws) == 580
    r = ref.beam_select(x.double().cpu().numpy(), s.astype(np.float64), n_out, temperature=temperature)
    for k in ("parent", "token"):
        np.testing.assert_array_equal(o[k].cpu().numpy(), r[k], err_msg=k)
    big = 2.0 ** -51 * float(x.double().abs().max()) / temperature
    for got, want in ((o["score"].cpu().numpy(), r["score"]), (lse.cpu().numpy(), r["lse"])):
        with np.errstate(over="ignore"):
            f = want.astype(np.float32).astype(np.float64)             # (a float may hold no more than infinity)
        fin = np.isfinite(f)
        np.testing.assert_array_equal(got[~fin], f[~fin])
        assert (np.abs(got[fin] - want[fin]) <= 2.0 ** -24 * np.abs(want[fin]) + 3e-6 + big).all()


@pytest.mark.parametrize("V", [50, 5000])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 2.0 ** -20, 2.0 ** 10])
@pytest.mark.parametrize("base", [1e6, 1e8, 3e8, 7.4e8, 7.5e8, 1e9, 1.4e9, 1e10, 1e12, 1e20, 1e30, 3e38])
def test_fp32_rows_about_a_large_logit(L, base, temperature, V):
    """A few neighbouring floats about +base and -base, many of each."""
    rng = np.random.default_rng([V, int(np.log10(base) * 10)])
    for sign in (1.0, -1.0):
        x = np.full((2, V), sign * base, np.float32)
        steps = rng.integers(0, 40, (2, V))
        x += steps * np.spacing(np.float32(base) / 2) * (1 if base < 1e38 else 0)
        check(L, torch.from_numpy(x.astype(np.float32)).cuda(), 6, temperature)
        x[:, V // 2] += np.spacing(x[:, V // 2]) * 64 if base < 1e38 else 0.0
        x[1, :V // 3] = -np.inf
        check(L, torch.from_numpy(x.astype(np.float32)).cuda(), 6, temperature)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("temperature", [2.0 ** -10, 2.0 ** -24, 2.0 ** -30, 2.0 ** -60, 2.0 ** -99])
def test_small_temperatures(L, dtype, temperature):
    rng = np.random.default_rng(3)
    for V in (50, 9001):
        x = torch.from_numpy(rng.standard_normal((2, V)).astype(np.float32) * 3).cuda().to(DTYPES[dtype])
        check(L, x, 5, temperature)
        check(L, x + 20, 5, temperature)


@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e30, float(np.finfo(np.float32).min)])
def test_a_row_masked_by_adding(L, mask):
    """Everything at the mask's value, with the logits under it or lost in it; a row with a few left."""
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((2, 4003)) * 3).astype(np.float32)
    m = np.float32(mask) + (x if mask > -1e38 else 0 * x)
    check(L, torch.from_numpy(m).cuda(), 6, 1.0)
    m[0, [5, 900, 4002]] = x[0, [5, 900, 4002]]
    check(L, torch.from_numpy(m).cuda(), 6, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("temperature", [0.7, 1.0, 3.0, 1000.0, 1e-4])
@pytest.mark.parametrize("V", [1, 3, 700, 20011])
def test_beams_of_which_everything_is_masked(L, dtype, temperature, V):
    """A row whose every logit is the type's lowest value (or -1e30): its log-sum-exp is that value, in a double, and
    its scores are the beam's, beside those of ordinary rows."""
    rng = np.random.default_rng(V)
    K = 6
    x = (rng.standard_normal((K, V)) * 3).astype(np.float32)
    low = torch.finfo(DTYPES[dtype]).min
    x[1] = low
    x[3] = low if dtype == "f16" else -1e30
    x[4, V // 2:] = low
    x = torch.from_numpy(x).cuda().to(DTYPES[dtype])
    s = -np.linspace(0.5, 3.0, K).astype(np.float32)[None]
    n = min(2 * K, K * V)
    ws = L.decode_workspace(L.KIND_BEAM_SELECT, 1, K, V, n)
    o = L.lossk_beam_select(x, torch.from_numpy(s).cuda(), n, temperature=temperature, ws=ws)
    assert L.lossk_device_status(ws) == 580
    r = ref.beam_select(x.double().cpu().numpy(), s.astype(np.float64), n, temperature=temperature)
    got, want = o["score"].cpu().numpy(), r["score"]
    with np.errstate(over="ignore"):
        want = np.where(np.isinf(want.astype(np.float32)), -np.inf, want)
    fin = np.isfinite(want)
    assert (got[~fin] == -np.inf).all()
    # (2^-51: of 65504 / T the doubles' own steps; of the lowest fp32 and bf16 values no step may be seen)
    bound = 2.0 ** -24 * np.abs(want[fin]) + 3e-6 + 2.0 ** -51 * 65504 / temperature
    assert (np.abs(got[fin] - want[fin]) <= bound).all()
    for k in ("parent", "token"):
        np.testing.assert_array_equal(o[k].cpu().numpy(), r[k], err_msg=k)
