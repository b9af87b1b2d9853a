"""Beam selection and state reordering on the GPU against plain 64-bit definitions.

Scores: the output rounds to float (half a step, 2^-24 of the value); before that the log-sum-exp
carries each exponential's error -- at most 2 steps of 2^-23 of its own plus the rounding of its
argument, 2^-24 of up to 40 in log2 units times ln 2 -- under 3e-6 in all.
"""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS, LSE = 2.0 ** -24, 3e-6


@pytest.fixture(scope="module")
def L():
    from conftest import build_lib
    build_lib()
    import output_projection_cross_gb300 as L
    assert torch.cuda.is_available()
    return L


def check(L, x, scores, n_out, status=580, allow=None, **kw):
    """x: GPU logits; scores, finished, lengths: numpy; allow: numpy int32 words [1 or rows][words]."""
    rows, V = x.shape
    g = {k: (torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v) for k, v in kw.items()}
    B, K = scores.shape
    ws = L.decode_workspace(L.KIND_BEAM_SELECT, B, K, V, n_out)
    lse = torch.full((rows,), 7.0, device="cuda")
    o = L.lossk_beam_select(x, torch.from_numpy(scores).cuda(), n_out, lse_out=lse, ws=ws,
                            allow=None if allow is None else torch.from_numpy(allow).cuda(), **g)
    assert L.lossk_device_status(ws) == status
    bits = None if allow is None else np.broadcast_to(ref.allowed_bits(allow, V), (rows, V))
    r = ref.beam_select(x.double().cpu().numpy(), scores.astype(np.float64), n_out, allow=bits, **kw)
    got = {k: v.cpu().numpy() for k, v in o.items()}
    for k in ("parent", "token", "finished", "length"):
        np.testing.assert_array_equal(got[k], r[k], err_msg=k)
    for k, v in (("score", got["score"]), ("lse", lse.cpu().numpy())):
        fin = np.isfinite(r[k])
        np.testing.assert_array_equal(fin, np.isfinite(v), err_msg=k)
        assert (v[~fin] == -np.inf).all()
        assert (np.abs(v[fin] - r[k][fin]) <= EPS * np.abs(r[k][fin]) + LSE).all(), k
    return got


def logits(rng, rows, V, dtype, scale=2.5):
    x = rng.standard_normal((rows, V)).astype(np.float32) * scale
    return torch.from_numpy(x).cuda().to(DTYPES[dtype])


def start(rng, B, K):
    return -(rng.random((B, K)) * 5 + 0.1).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,K,V,n_out", [
    (1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 2, 6), (3, 4, 7, 8), (1, 1, 31, 1), (2, 2, 33, 4), (1, 64, 65, 128),
    (5, 7, 1001, 14), (1, 4, 4097, 128), (2, 16, 8200, 32), (1, 4, 50021, 8), (40, 2, 999, 3)])
def test_select(L, dtype, B, K, V, n_out):
    rng = np.random.default_rng([B, K, V, n_out])
    check(L, logits(rng, B * K, V, dtype), start(rng, B, K), n_out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_large_vocabulary(L, dtype):
    rng = np.random.default_rng(5)
    check(L, logits(rng, 6, 151936, dtype), start(rng, 2, 3), 12, temperature=0.8)


@pytest.mark.parametrize("V", [5, 64, 1000, 20011])
def test_select_ties_go_to_the_lowest(L, V):
    """Constant rows, and identical beams: every comparison is a tie."""
    x = torch.zeros(6, V, device="cuda", dtype=torch.bfloat16)
    s = np.zeros((2, 3), np.float32)
    got = check(L, x, s, 16)
    n = min(16, 3 * V)
    flat = got["parent"][0, :n].astype(np.int64) * V + got["token"][0, :n]
    assert flat.tolist() == sorted(flat.tolist())
    rng = np.random.default_rng(V)
    one = logits(rng, 1, V, "bf16", 1.0)
    check(L, one.expand(6, V).contiguous(), s, 16)
    # few distinct values, many ties inside a row
    x = torch.from_numpy(rng.integers(-2, 3, (6, V)).astype(np.float32)).cuda()
    check(L, x, start(rng, 2, 3), 16)


def test_select_negative_zero_ties_with_zero(L):
    x = torch.full((1, 4000), -1.0, device="cuda")
    x[0, 100], x[0, 7], x[0, 3000] = 0.0, -0.0, 0.0
    assert check(L, x, np.zeros((1, 1), np.float32), 3)["token"].tolist() == [[7, 100, 3000]]


@pytest.mark.parametrize("order", ["rising", "falling", "spike"])
def test_select_orders_that_defeat_a_threshold(L, order):
    V = 30000
    x = np.arange(V, dtype=np.float32)[None] * 1e-3
    if order == "falling":
        x = x[:, ::-1]
    if order == "spike":
        x = np.where(np.arange(V)[None] % 997 == 5, 9.0 + x, 0.0).astype(np.float32)
    x = torch.from_numpy(np.repeat(x, 2, 0).copy()).cuda()
    check(L, x, np.array([[-0.3, -0.9]], np.float32), 128)


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 37, 5003, 40000])
def test_select_allowed_tokens(L, dtype, V, shared):
    """A bit mask; what the logits hold where it says no does not matter."""
    rng = np.random.default_rng([V, shared])
    rows = 6
    words = (V + 31) // 32
    bits = rng.integers(0, 1 << 32, (1 if shared else rows, words), dtype=np.uint64).astype(np.uint32)
    if not shared:
        bits[2] = 0                                    # one beam may go nowhere
        bits[3] = 0
        bits[3, V // 64] = 1 << (V // 2 % 32)          # one has a single way
    allow = bits.view(np.int32)
    x = logits(rng, rows, V, dtype)
    off = torch.from_numpy(~np.broadcast_to(ref.allowed_bits(allow, V), (rows, V))).cuda()
    for junk in (float("nan"), float("inf"), -float("inf"), torch.finfo(x.dtype).min):
        check(L, torch.where(off, torch.tensor(junk, device="cuda", dtype=x.dtype), x).contiguous(), start(rng, 2, 3), 10,
              allow=allow)
    # another alignment of rows: a view whose rows are wider than the vocabulary
    wide = torch.full((rows, V + 24), float("nan"), device="cuda", dtype=x.dtype)
    wide[:, :V] = x
    check(L, wide[:, :V], start(rng, 2, 3), 10, allow=allow)


def test_select_masked_logits(L):
    """-infinity is no candidate; a row of nothing else has none; the type's lowest value is one."""
    rng = np.random.default_rng(11)
    x = logits(rng, 8, 3001, "f32")
    x[0, :] = -float("inf")
    x[1, 1:] = -float("inf")
    x[2, :] = torch.finfo(torch.float32).min
    x[3, 5:] = torch.finfo(torch.float32).min
    s = np.array([[-1, -2, -3, -np.inf], [-np.inf] * 4], np.float32)
    got = check(L, x, s, 8)
    assert (got["parent"][1] == -1).all()
    x[:, :] = -float("inf")
    assert (check(L, x, np.zeros((2, 4), np.float32), 8)["token"] == -1).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 1500, 3000])
def test_select_reports_logits_that_are_not_numbers(L, what, at):
    rng = np.random.default_rng(12)
    x = logits(rng, 4, 3001, "bf16")
    x[1, at] = what
    check(L, x, start(rng, 1, 4), 6, status=585)
    s = start(rng, 1, 4)
    s[0, 2] = what
    check(L, logits(rng, 4, 3001, "bf16"), s, 6, status=585)


@pytest.mark.parametrize("alpha", [0.0, 0.6, 1.0, -0.5])
def test_select_finished_beams_and_lengths(L, alpha):
    """A finished beam stands for itself; its logits are not read (here they are NaN)."""
    rng = np.random.default_rng(13)
    B, K, V = 5, 6, 2003
    x = logits(rng, B * K, V, "bf16")
    fin = (rng.random((B, K)) < 0.4).astype(np.uint8)
    fin[0], fin[1] = 1, 0
    x[torch.from_numpy(fin.reshape(-1).astype(bool)).cuda()] = float("nan")
    ln = rng.integers(0, 60, (B, K)).astype(np.int32)
    for end in (0, 1234, V - 1, -1):
        if end >= 0:
            x[:, end] += 4.0                           # hypotheses that end are among the chosen
        check(L, x, start(rng, B, K), 2 * K, finished=fin, end_token=end, lengths=ln, length_alpha=alpha)
    check(L, x, start(rng, B, K), 3, finished=fin, end_token=7)


def test_select_first_step(L):
    """All beams of an entry alike, all but the first dead: how a search starts."""
    rng = np.random.default_rng(14)
    x = logits(rng, 2, 9001, "f16").repeat_interleave(4, 0).contiguous()
    s = np.full((2, 4), -np.inf, np.float32)
    s[:, 0] = 0.0
    got = check(L, x, s, 4)
    assert (got["parent"] == 0).all()


def test_select_repeats_bit_for_bit_and_on_another_stream(L):
    rng = np.random.default_rng(15)
    x = logits(rng, 32, 60013, "bf16")
    s = torch.from_numpy(start(rng, 8, 4)).cuda()
    a = L.lossk_beam_select(x, s, 8)
    a = {k: v.clone() for k, v in a.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            b = L.lossk_beam_select(x, s, 8)
        side.synchronize()
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_select_in_a_graph(L):
    rng = np.random.default_rng(16)
    x, s = logits(rng, 8, 20001, "bf16"), torch.from_numpy(start(rng, 2, 4)).cuda()
    ws = L.decode_workspace(L.KIND_BEAM_SELECT, 2, 4, 20001, 8)
    o = L.beam_buffers(2, 8)
    L.lossk_beam_select(x, s, 8, out=o, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lossk_beam_select(x, s, 8, out=o, ws=ws)
    for i in range(3):
        x.copy_(logits(rng, 8, 20001, "bf16"))
        g.replay()
        torch.cuda.synchronize()
        r = ref.beam_select(x.double().cpu().numpy(), s.double().cpu().numpy(), 8)
        np.testing.assert_array_equal(o["token"].cpu().numpy(), r["token"])
        np.testing.assert_array_equal(o["parent"].cpu().numpy(), r["parent"])


def test_select_binding_refuses(L):
    x = torch.zeros(4, 10, device="cuda")
    s = torch.zeros(2, 2, device="cuda")
    with pytest.raises(ValueError):
        L.lossk_beam_select(x, s[:1], 2)
    with pytest.raises(TypeError):
        L.lossk_beam_select(x, s.double(), 2)
    with pytest.raises(TypeError):
        L.lossk_beam_select(x.to(torch.int32), s, 2)
    with pytest.raises(ValueError):
        L.lossk_beam_select(x, s, 2, allow=torch.zeros(3, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        L.lossk_beam_select(x.T.contiguous().T, s, 2)
    with pytest.raises(L.LosskError) as e:
        L.lossk_beam_select(x, s, 2, end_token=10)
    assert e.value.status == 586


@pytest.mark.parametrize("shape,dtype", [((1,), torch.uint8), ((3,), torch.int32), ((5, 7), torch.bfloat16),
                                         ((16,), torch.float32), ((70001,), torch.uint8), ((300, 1024), torch.bfloat16)])
def test_gather(L, shape, dtype):
    rng = np.random.default_rng(17)
    G, n_src, n_dst = 3, 4, 6
    src = torch.from_numpy(rng.integers(0, 100, (G, n_src) + shape)).cuda().to(dtype)
    par = torch.from_numpy(rng.integers(-1, n_src, (G, n_dst)).astype(np.int32)).cuda()
    dst = L.lossk_beam_gather(src, par)
    want = torch.stack([torch.stack([src[g, p] if p >= 0 else torch.zeros_like(src[0, 0]) for p in par[g].tolist()])
                        for g in range(G)])
    assert torch.equal(dst, want)


def test_gather_reports_a_bad_parent(L):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    src = torch.ones(2, 3, 8, device="cuda")
    for bad in (3, -2, 1 << 30):
        par = torch.tensor([[0, bad], [1, 2]], dtype=torch.int32, device="cuda")
        d = L.lossk_beam_gather(src, par, ws=ws)
        assert L.lossk_device_status(ws) == 586
        assert L.lossk_device_status(ws) == 580
        assert d[0, 1].abs().sum() == 0 and d[0, 0].sum() == 8
