"""Attention over a paged cache on the GPU against a plain 64-bit one.

An output is the weighted mean of values: its rounding to the type is half a step (eps / 2) of
itself; what the fp32 sums before it add is bounded by the same mean over |v|: each weight's
exponent carries the rounding of a dot product of hd terms, at most 2^-24 (hd + 8) sum|q k| scale
(with |x| there below 40 by the inputs' sizes), each exponential 2 steps of 2^-23, the sums over
n tokens a few more.  The tests' bound: eps / 2 |out| + 2^-24 (40 (hd / 8 + 8) + 64) mean|v|,
where hd / 8 stands for hd terms of random sign added in blocks.  lse: 2^-24 of itself and of
the exponents' error.
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


def cache(rng, lens, page, kv, hd, dtype, share=1, prefix=0, junk=float("nan"), layout="token", spare=3):
    """Pages for sequences of these lengths, groups of `share` sharing their first `prefix` pages;
    what no token covers holds junk.  Returns k, v (views [pages][page][kv][hd]) and the table."""
    S = len(lens)
    used = [-(-n // page) for n in lens]
    rows, nxt = [], 0
    for s in range(S):
        pre = min([prefix] + [lens[i] // page for i in range(s // share * share, s // share * share + share)]) \
            if share > 1 else 0
        own = list(range(nxt, nxt + used[s] - (pre if s % share else 0)))
        nxt += len(own)
        rows.append((rows[s // share * share][:pre] if s % share else []) + own)
    n_pages = nxt + spare
    perm = rng.permutation(n_pages)
    m = max(1, max(used))
    table = np.full((S, m), -1, np.int32)
    kv_ = np.full((2, n_pages, page, kv, hd), junk, np.float32)
    for s, r in enumerate(rows):
        table[s, :used[s]] = perm[np.array(r, np.int64)] if r else []
        for c in range(used[s]):
            n = min(page, lens[s] - c * page)
            kv_[:, table[s, c], :n] = rng.standard_normal((2, n, kv, hd))
    t = torch.from_numpy(kv_).to(DTYPES[dtype]).cuda()
    if layout == "head":
        t = t.transpose(2, 3).contiguous().transpose(2, 3)
    return t[0], t[1], table


def check(L, rng, lens, hq, kv, hd, page=16, dtype="bf16", window=0, scale=None, status=580, q=None, kvt=None, **c):
    S = len(lens)
    share = c.get("share", 1)
    k, v, table = kvt if kvt is not None else cache(rng, lens, page, kv, hd, dtype, **c)
    if q is None:
        q = torch.from_numpy(rng.standard_normal((S, hq, hd)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    ws = L.decode_workspace(L.KIND_PAGED_ATTN, S, hq, kv, hd)
    lse = torch.full((S, hq), 7.0, device="cuda")
    out = L.lossk_paged_attn(q, k, v, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             scale=scale, window=window, share=share, lse_out=lse, ws=ws)
    assert L.lossk_device_status(ws) == status
    sc = hd ** -0.5 if scale is None else scale
    qd, kd, vd = (t.double().cpu().numpy() for t in (q, k, v))
    r, rl = ref.attend(qd, kd, vd, table, lens, page, sc, window)
    mean, _ = ref.attend(qd, kd, np.abs(vd), table, lens, page, sc, window)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    eps = torch.finfo(DTYPES[dtype]).eps
    x_err = 2.0 ** -24 * (40 * (hd / 8 + 8) + 64)
    assert np.isfinite(got).all()
    assert (np.abs(got - r) <= eps / 2 * np.abs(r) + x_err * mean + (2.0 ** -24 if dtype == "f16" else 0)).all(), \
        np.abs(got - r).max()
    fin = np.isfinite(rl)
    assert (gl[~fin] == -np.inf).all() and (np.abs(gl - rl)[fin] <= 2.0 ** -24 * np.abs(rl[fin]) + x_err).all()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,kv,hd", [(1, 1, 8), (4, 4, 32), (8, 2, 64), (6, 2, 72), (5, 1, 80), (16, 2, 96),
                                      (8, 1, 128), (16, 1, 128), (34, 2, 128), (3, 3, 136), (8, 2, 192), (40, 1, 200),
                                      (12, 3, 256)])
def test_heads(L, dtype, hq, kv, hd):
    rng = np.random.default_rng([hq, kv, hd])
    check(L, rng, [1, 0, 37, 16, 300], hq, kv, hd, dtype=dtype)


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("page", [1, 3, 16, 32, 100, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages(L, dtype, page, layout):
    rng = np.random.default_rng(page)
    check(L, rng, [0, 1, 15, 16, 17, 31, 32, 33, 64, 99, 100, 101, 255, 256, 257, 511, 700], 4, 2, 64, page=page,
          dtype=dtype, layout=layout)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[0], [1], [2], [5000], [0, 0, 0], [0, 3000, 0, 1], [1] * 70, [40000, 1, 17]])
def test_lengths(L, dtype, lens):
    rng = np.random.default_rng(len(lens))
    check(L, rng, lens, 8, 2, 128, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("window", [1, 5, 16, 33, 1000, 1 << 40])
def test_window(L, dtype, window):
    rng = np.random.default_rng(7)
    check(L, rng, [0, 1, 5, 6, 32, 33, 34, 200, 1500], 6, 2, 64, dtype=dtype, window=min(window, 1 << 29))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("share,hq,kv,hd", [(2, 2, 2, 64), (3, 6, 2, 128), (8, 8, 2, 128), (5, 7, 1, 96),
                                            (10, 32, 2, 64), (4, 4, 2, 200)])
@pytest.mark.parametrize("prefix", [0, 1, 9, 1000])
def test_beams_that_share_pages(L, dtype, share, hq, kv, hd, prefix):
    rng = np.random.default_rng([share, prefix])
    lens = [200 + i for i in range(share)] + [150] * share + [0] * share + [15] * share
    check(L, rng, lens, hq, kv, hd, dtype=dtype, share=share, prefix=prefix)


@pytest.mark.parametrize("window", [1, 20, 100, 149, 150, 400])
def test_beams_that_share_pages_under_a_window(L, window):
    rng = np.random.default_rng(window)
    lens = [150] * 4 + [160, 150, 155, 151] + [16] * 4
    check(L, rng, lens, 8, 2, 64, share=4, prefix=6, window=window)


def test_sharing_changes_only_rounding(L):
    rng = np.random.default_rng(8)
    lens = [1000 + i for i in range(8)]
    kvt = cache(rng, lens, 16, 2, 128, "f32", share=8, prefix=50)
    q = torch.from_numpy(rng.standard_normal((8, 8, 128)).astype(np.float32)).cuda()
    a = check(L, rng, lens, 8, 2, 128, dtype="f32", q=q, kvt=kvt, share=8)
    b = check(L, rng, lens, 8, 2, 128, dtype="f32", q=q, kvt=kvt)
    assert (a - b).abs().max() < 1e-5


def test_pages_shared_by_sequences_that_are_no_group(L):
    rng = np.random.default_rng(9)
    k, v, table = cache(rng, [64, 64, 64, 64], 16, 2, 64, "bf16")
    table[2, :3], table[3, 0] = table[0, :3], table[1, 0]
    check(L, rng, [64] * 4, 4, 2, 64, kvt=(k, v, table))
    check(L, rng, [64] * 4, 4, 2, 64, kvt=(k, v, table), share=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(L, dtype):
    """Exponents that a softmax without its maximum would not survive; a maximum that keeps rising."""
    rng = np.random.default_rng(10)
    n, hd = 700, 64
    k, v, table = cache(rng, [n, n], 16, 1, hd, dtype)
    for s in range(2):
        for j in range(n):
            k[table[s, j // 16], j % 16, 0, 0] = (j if s == 0 else n - j) * 0.25
    q = torch.zeros((2, 2, hd), device="cuda", dtype=DTYPES[dtype])
    q[:, 0, 0], q[:, 1, 0] = 4.0, -4.0
    out = L.lossk_paged_attn(q, k, v, torch.from_numpy(table).cuda(), torch.tensor([n, n], dtype=torch.int32).cuda(),
                             scale=1.0)
    r, _ = ref.attend(*(t.double().cpu().numpy() for t in (q, k, v)), table, [n, n], 16, 1.0)
    eps = torch.finfo(DTYPES[dtype]).eps
    # products up to 700 are exact here; an exponent's rounding is 2^-24 of 1010
    assert (np.abs(out.double().cpu().numpy() - r) <= eps / 2 * np.abs(r) + 2.0 ** -24 * 1500 * np.abs(r).max()).all()


@pytest.mark.parametrize("junk", [0.0, float("nan"), float("inf"), -float("inf"), 1e4])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_what_lies_past_the_end_does_not_matter(L, dtype, junk):
    rng = np.random.default_rng(11)
    check(L, rng, [1, 17, 33, 47], 4, 2, 64, page=64, dtype=dtype, junk=junk)
    check(L, rng, [1, 17, 33, 47], 4, 2, 64, page=64, dtype=dtype, junk=junk, window=9)


def test_a_fused_projection_slice(L):
    """q as a part of wider rows; pages of one layer out of a pool of several."""
    rng = np.random.default_rng(12)
    S, hq, kv, hd = 5, 4, 2, 64
    lens = [3, 50, 16, 0, 77]
    k, v, table = cache(rng, lens, 16, kv, hd, "bf16")
    pool = torch.full((3, 2) + tuple(k.shape), float("nan"), device="cuda", dtype=torch.bfloat16)
    pool[1, 0], pool[1, 1] = k, v
    wide = torch.randn((S, (hq + 2 * kv) * hd), device="cuda").bfloat16()
    check(L, rng, lens, hq, kv, hd, q=wide[:, :hq * hd].unflatten(1, (hq, hd)), kvt=(pool[1, 0], pool[1, 1], table))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ids_and_lengths_out_of_range(L, dtype):
    rng = np.random.default_rng(13)
    lens = [40, 64, 20]
    k, v, table = cache(rng, lens, 16, 2, 64, dtype)
    q = torch.from_numpy(rng.standard_normal((3, 4, 64)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    good = check(L, rng, lens, 4, 2, 64, dtype=dtype, q=q, kvt=(k, v, table))
    ws = L.decode_workspace(L.KIND_PAGED_ATTN, 3, 4, 2, 64)
    for bad in (k.shape[0], -1, 1 << 30):
        t = table.copy()
        t[1, 2] = bad
        out = L.lossk_paged_attn(q, k, v, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 ws=ws)
        assert L.lossk_device_status(ws) == 586 and L.lossk_device_status(ws) == 580
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        # the page's tokens are left out: attention over the other three pages
        kept = np.delete(table, 2, 1)
        r, _ = ref.attend(*(x.double().cpu().numpy() for x in (q, k, v)), kept, [0, 48, 0], 16, 0.125)
        eps = torch.finfo(DTYPES[dtype]).eps
        assert (np.abs(out[1].double().cpu().numpy() - r[1]) <= eps / 2 * np.abs(r[1]) + 5e-5).all()
    for bad in (65, -1, 1 << 30):
        out = L.lossk_paged_attn(q, k, v, torch.from_numpy(table).cuda(),
                                 torch.tensor([40, bad, 20], dtype=torch.int32).cuda(), ws=ws)
        assert L.lossk_device_status(ws) == 586
        assert out[1].abs().max() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_again_and_on_another_stream(L, dtype):
    rng = np.random.default_rng(14)
    lens = [3000, 1, 500, 77]
    kvt = cache(rng, lens, 16, 4, 128, dtype)
    q = torch.from_numpy(rng.standard_normal((4, 16, 128)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    a = check(L, rng, lens, 16, 4, 128, dtype=dtype, q=q, kvt=kvt)
    t, n = torch.from_numpy(kvt[2]).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ws = L.decode_workspace(L.KIND_PAGED_ATTN, 4, 16, 4, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            b = L.lossk_paged_attn(q, kvt[0], kvt[1], t, n, ws=ws)
        side.synchronize()
        assert torch.equal(a, b)


def test_in_a_graph_with_lengths_that_grow(L):
    rng = np.random.default_rng(15)
    kvt = cache(rng, [120, 90], 16, 2, 64, "bf16")
    q = torch.randn((2, 4, 64), device="cuda").bfloat16()
    t, n = torch.from_numpy(kvt[2]).cuda(), torch.tensor([40, 3], dtype=torch.int32).cuda()
    ws, out = L.decode_workspace(L.KIND_PAGED_ATTN, 2, 4, 2, 64), torch.empty_like(q)
    L.lossk_paged_attn(q, kvt[0], kvt[1], t, n, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lossk_paged_attn(q, kvt[0], kvt[1], t, n, out=out, ws=ws)
    for a, b in ((40, 3), (41, 90), (120, 0)):
        n.copy_(torch.tensor([a, b], dtype=torch.int32))
        g.replay()
        want = L.lossk_paged_attn(q, kvt[0], kvt[1], t, n)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_offsets_beyond_32_bits(L):
    """A cache of over 4 GiB a plane, its last pages in use."""
    rng = np.random.default_rng(16)
    n_pages, page, kv, hd = 1100, 64, 128, 256
    big = torch.empty((2, n_pages, page, kv, hd), device="cuda", dtype=torch.bfloat16)
    assert big[0].numel() * 2 > 1 << 32
    table = np.array([[n_pages - 1, n_pages - 3]], np.int32)
    for p in table[0]:
        big[:, p] = torch.randn((2, page, kv, hd), device="cuda").bfloat16()
    q = torch.randn((1, kv, hd), device="cuda").bfloat16()
    out = L.lossk_paged_attn(q, big[0], big[1], torch.from_numpy(table).cuda(),
                             torch.tensor([100], dtype=torch.int32).cuda())
    small = big[:, [n_pages - 1, n_pages - 3]].double().cpu().numpy()
    r, _ = ref.attend(q.double().cpu().numpy(), small[0], small[1], np.array([[0, 1]]), [100], page, hd ** -0.5)
    assert (np.abs(out.double().cpu().numpy() - r) <= 2.0 ** -8 * np.abs(r) + 2e-4).all()


def test_binding_refuses(L):
    k = torch.zeros((4, 16, 2, 64), device="cuda", dtype=torch.bfloat16)
    t = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros((2, 4, 64), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        L.lossk_paged_attn(q.half(), k, k, t, n)
    with pytest.raises(ValueError):
        L.lossk_paged_attn(q[:1], k, k, t, n)
    with pytest.raises(ValueError):
        L.lossk_paged_attn(q, k, k[:, :8], t, n)
    with pytest.raises(TypeError):
        L.lossk_paged_attn(q, k, k, t.long(), n)
    with pytest.raises(L.LosskError) as e:
        L.lossk_paged_attn(q, k, k, t, n, share=3)
    assert e.value.status == 582
