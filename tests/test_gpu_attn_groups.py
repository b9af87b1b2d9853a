"""Attention over a paged cache for more sequences than the split pass's blocks sum up for themselves (1024
groups), alone and in groups that share pages; what such calls launch."""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PAGE, KV, HD = 4, 2, 64


@pytest.fixture(scope="module")
def L():
    from conftest import build_lib
    build_lib()
    import output_projection_cross_gb300 as L
    assert torch.cuda.is_available()
    return L


@pytest.mark.parametrize("groups,share,launches", [(3, 1, 2), (3, 2, 3), (1024, 1, 2), (1024, 2, 3), (1025, 1, 3),
                                                   (1025, 2, 4)])
def test_kernels_counted(L, groups, share, launches):
    S = groups * share
    k = torch.randn(4, PAGE, KV, HD, device="cuda").bfloat16()
    q = torch.randn(S, KV, HD, device="cuda").bfloat16()
    table, lens = torch.zeros(S, 1, dtype=torch.int32, device="cuda"), torch.full((S,), 3, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    before = L.lossk_launch_count()
    L.lossk_paged_attn(q, k, k, table, lens, share=share)
    assert L.lossk_launch_count() - before == launches


def cache(rng, lens, share, dtype):
    """Pages of sequences of these lengths; groups share the first two pages that all of their rows fill.
    (Bounds as in test_gpu_attn.py.)"""
    S = len(lens)
    used = [-(-n // PAGE) for n in lens]
    rows, nxt = [], 0
    for s in range(S):
        first = s // share * share
        pre = min([2] + [lens[i] // PAGE for i in range(first, first + share)]) if share > 1 else 0
        own = list(range(nxt, nxt + used[s] - (pre if s % share else 0)))
        nxt += len(own)
        rows.append((rows[first][:pre] if s % share else []) + own)
    perm = rng.permutation(nxt + 3)
    table = np.full((S, max(1, max(used))), -1, np.int32)
    for s, r in enumerate(rows):
        table[s, :len(r)] = perm[np.array(r, np.int64)] if r else []
    kv = rng.standard_normal((2, nxt + 3, PAGE, KV, HD)).astype(np.float32)
    t = torch.from_numpy(kv).to(DTYPES[dtype]).cuda()
    return t[0], t[1], table


def compare(L, q, k, v, table, lens, dtype, share=1, window=0, status=580):
    S, hq = q.shape[:2]
    ws = L.decode_workspace(L.KIND_PAGED_ATTN, S, hq, KV, HD)
    lse = torch.full((S, hq), 7.0, device="cuda")
    out = L.lossk_paged_attn(q, k, v, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             share=share, window=window, lse_out=lse, ws=ws)
    assert L.lossk_device_status(ws) == status
    limit = table.shape[1] * PAGE
    good = [n if 0 <= n <= limit else 0 for n in lens]
    qd, kd, vd = (t.double().cpu().numpy() for t in (q, k, v))
    r, rl = ref.attend(qd, kd, vd, table, good, PAGE, HD ** -0.5, window)
    mean, _ = ref.attend(qd, kd, np.abs(vd), table, good, PAGE, HD ** -0.5, window)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    x_err = 2.0 ** -24 * (40 * (HD / 8 + 8) + 64)
    bound = torch.finfo(DTYPES[dtype]).eps / 2 * np.abs(r) + x_err * mean + (2.0 ** -24 if dtype == "f16" else 0)
    assert (np.abs(got - r) <= bound).all()
    fin = np.isfinite(rl)
    assert (gl[~fin] == -np.inf).all()
    assert (np.abs(gl[fin] - rl[fin]) <= 2.0 ** -24 * np.abs(rl[fin]) + x_err).all()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("share", [1, 2, 3])
@pytest.mark.parametrize("groups", [1023, 1024, 1025, 2500])
def test_many_groups(L, dtype, share, groups):
    rng = np.random.default_rng([groups, share])
    S = groups * share
    lens = [int(n) for n in rng.integers(0, 20, S)]
    lens[7], lens[S - 1] = 700, 300                    # a few that are cut over many runs
    k, v, table = cache(rng, lens, share, dtype)
    q = torch.from_numpy(rng.standard_normal((S, 2 * KV, HD)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    out = compare(L, q, k, v, table, lens, dtype, share)
    again = compare(L, q, k, v, table, lens, dtype, share)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share", [1, 2])
def test_many_groups_under_a_window_and_with_bad_lengths(L, dtype, share):
    rng = np.random.default_rng(5)
    S = 1200 * share
    lens = [int(n) for n in np.repeat(rng.integers(0, 40, 1200), share)]
    k, v, table = cache(rng, lens, share, dtype)
    q = torch.from_numpy(rng.standard_normal((S, KV, HD)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    compare(L, q, k, v, table, lens, dtype, share, window=9)
    for at, bad in ((0, -1), (S - 1, 41), (1100, 1 << 30)):
        lens[at] = bad
    compare(L, q, k, v, table, lens, dtype, share, status=586)


def test_all_empty(L):
    rng = np.random.default_rng(6)
    k, v, table = cache(rng, [1] * 1100, 1, "bf16")
    q = torch.from_numpy(rng.standard_normal((1100, KV, HD)).astype(np.float32)).bfloat16().cuda()
    assert compare(L, q, k, v, table, [0] * 1100, "bf16").abs().max() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [(1 << 30) - 1, 1 << 30, (1 << 31) + 5, 1 << 40])
def test_windows_wider_than_any_sequence(L, dtype, window):
    rng = np.random.default_rng(7)
    lens = [0, 1, 33, 200, 1500]
    k, v, table = cache(rng, lens, 1, dtype)
    q = torch.from_numpy(rng.standard_normal((5, 2 * KV, HD)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    a = compare(L, q, k, v, table, lens, dtype, window=window)
    assert torch.equal(a, compare(L, q, k, v, table, lens, dtype))
