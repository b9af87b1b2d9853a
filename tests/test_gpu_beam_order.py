"""The order of candidates where their ranks meet."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from conftest import build_lib
    build_lib()
    import output_projection_cross_gb300 as L
    assert torch.cuda.is_available()
    return L


def finished(L, scores, lengths, alpha, n_out=None):
    """Parents in order, of beams that are all finished: rank = score / length ^ alpha."""
    s = torch.tensor([scores], dtype=torch.float32, device="cuda")
    K = s.shape[1]
    o = L.lossk_beam_select(torch.zeros(K, 10, device="cuda"), s, n_out or K,
                            finished=torch.ones(1, K, dtype=torch.uint8, device="cuda"), end_token=3,
                            lengths=torch.tensor([lengths], dtype=torch.int32, device="cuda"), length_alpha=alpha)
    return o["parent"][0].tolist()


def test_equal_quotients_go_to_the_lower_beam(L):
    """n scores of -r n over lengths n are one rank; with the product by 1 / n instead of the quotient
    those of n = 49, 98, 103 ... lie a step beside it."""
    for r in (1.0, 3.0, 0.37109375):
        for at in range(1, 1000, 60):
            n = list(range(at, at + 60))
            for order in (n, n[::-1]):
                assert finished(L, [-r * x for x in order], order, 1.0) == list(range(60))
    squares = [k * k for k in range(1, 61)]            # and of the square root of perfect squares
    assert finished(L, [-float(k) for k in range(1, 61)], squares, 0.5) == list(range(60))
    assert finished(L, [-float(k) for k in range(60, 0, -1)], squares[::-1], 0.5) == list(range(60))
    assert finished(L, [-float(k * k) for k in range(1, 61)], list(range(1, 61)), 2.0) == list(range(60))


@pytest.mark.parametrize("alpha", [0.6, 1.0, -0.5, 2.0, 1e3, -1e3])
def test_ranks_of_many_lengths(L, alpha):
    rng = np.random.default_rng(1)
    for _ in range(20):
        s, n = -rng.random(40).astype(np.float32) * 30 - 0.1, rng.integers(0, 300, 40)
        with np.errstate(over="ignore", divide="ignore"):
            rank = [float(np.float64(x) / np.float64(max(1, m)) ** np.float64(alpha)) for x, m in zip(s, n)]
        want = sorted(range(40), key=lambda k: (-rank[k], k))
        got = finished(L, s.tolist(), n.tolist(), alpha)
        # (powers may differ in their last bit: ranks that close may stand in either order)
        assert sorted(got) == list(range(40))
        assert all(a == b or math.isclose(rank[a], rank[b], rel_tol=1e-15) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V", [40, 5003, 40000])
@pytest.mark.parametrize("temperature", [1e-30, 1e-6, 1e12, 1e20, 1e30])
def test_a_beam_s_candidates_are_in_the_order_of_their_logits(L, dtype, V, temperature):
    """At a high temperature different logits meet in one double: larger logits come first all the same, and of
    beams that are alike the lower one's candidates."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(1, V, device="cuda", generator=g).to(dtype).expand(3, V).contiguous()
    ws = L.decode_workspace(L.KIND_BEAM_SELECT, 1, 3, V, 12)
    o = L.lossk_beam_select(x, torch.tensor([[-1.0, -1.0, -2.0]], device="cuda"), 12, temperature=temperature, ws=ws)
    assert L.lossk_device_status(ws) == 580
    parent, token = o["parent"][0].tolist(), o["token"][0].tolist()
    f = x[0].double().cpu().numpy()
    best = sorted(range(V), key=lambda v: (-f[v], v))[:12]
    for k in range(3):
        mine = [v for p, v in zip(parent, token) if p == k]
        assert mine == best[:len(mine)]
    if temperature >= 1e20:                            # all of the first beam's ranks are one double, and the second's
        assert parent == [0] * 12
    elif temperature <= 1e-30:
        # only logits equal to the largest keep a score: then come, beam by beam, scores of -infinity's size
        ties = sum(1 for v in best if f[v] == f[best[0]])
        assert parent[:3 * ties] == ([0] * ties + [1] * ties + [2] * ties)[:12][:3 * ties]


def test_logits_closer_than_a_double_of_the_rank_resolves(L):
    x = torch.tensor([[0.0, 1e-30, 2e-30, 3e-30, -1e-30] + [-5.0] * 600], device="cuda")
    o = L.lossk_beam_select(x, torch.zeros(1, 1, device="cuda"), 4)
    assert o["token"].tolist() == [[3, 2, 1, 0]]
