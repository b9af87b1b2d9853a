"""Refusals and sizes of the decoding calls, on the CPU: every call below returns before its first
CUDA call (the addresses are made up and never followed)."""
import numpy as np
import pytest

P = 4096   # a made-up address, 256-byte aligned


@pytest.fixture(scope="module")
def L():
    from conftest import build_lib
    build_lib()
    import output_projection_cross_gb300 as L
    return L


def select_call(L, **over):
    a = dict(batch=2, beams=3, vocab=1000, n_out=6, dtype=1, logits=P, logits_len=6000, row_stride=1000, scores=P,
             scores_len=6, temperature=1.0, allow=None, allow_len=0, allow_stride=0, finished=None, end_token=-1,
             lengths=None, length_alpha=0.0, parent=P, token=P, score=P, finished_out=P, length_out=P, lse=None, ws=P,
             ws_bytes=1 << 24, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return L.lib.lossk_beam_select(*a.values())


def test_select_refusals(L):
    for size in ("batch", "beams", "vocab", "n_out"):
        assert select_call(L, **{size: 0}) == 581
        assert select_call(L, **{size: -3}) == 581
    assert select_call(L, beams=65) == 583
    assert select_call(L, n_out=129) == 583
    assert select_call(L, vocab=(1 << 24) + 1) == 583
    assert select_call(L, batch=(1 << 24) + 1) == 583
    for p in ("logits", "scores", "parent", "token", "score", "ws"):
        assert select_call(L, **{p: None}) == 582
    assert select_call(L, dtype=3) == 582
    assert select_call(L, logits_len=5999) == 582
    assert select_call(L, row_stride=999) == 582
    assert select_call(L, row_stride=1008) == 582            # six rows of that stride need 6040 elements
    assert select_call(L, scores_len=5) == 582
    assert select_call(L, allow=P, allow_len=31) == 582
    assert select_call(L, allow=P, allow_len=6 * 32, allow_stride=31) == 582
    assert select_call(L, allow=P, allow_len=6 * 32 - 1, allow_stride=32) == 582
    assert select_call(L, ws_bytes=L.lossk_decode_workspace_bytes(L.KIND_BEAM_SELECT, 2, 3, 1000, 6) - 1) == 582
    assert select_call(L, logits=P + 2) == 591
    assert select_call(L, ws=P + 16) == 591
    assert select_call(L, token=P + 4) == 591
    for t in (0.0, -1.0, float("nan"), float("inf")):
        assert select_call(L, temperature=t) == 585
    assert select_call(L, length_alpha=float("nan")) == 585
    assert select_call(L, end_token=-2) == 586
    assert select_call(L, end_token=1000) == 586


def test_select_check_order(L):
    assert select_call(L, batch=0, vocab=1 << 30, logits=None) == 581
    assert select_call(L, vocab=1 << 30, logits=None) == 583
    assert select_call(L, logits=None, temperature=0.0, ws=P + 1) == 582
    assert select_call(L, ws=P + 1, temperature=0.0) == 591
    assert select_call(L, temperature=0.0, end_token=5000) == 585


def gather_call(L, **over):
    a = dict(n_group=2, n_src=3, n_dst=4, row_bytes=40, parent=P, parent_len=8, src=P, src_bytes=240, dst=P,
             dst_bytes=320, ws=P, ws_bytes=256, stream=None)
    assert not set(over) - set(a)
    a.update(over)
    return L.lib.lossk_beam_gather(*a.values())


def test_gather_refusals(L):
    for size in ("n_group", "n_src", "n_dst", "row_bytes"):
        assert gather_call(L, **{size: 0}) == 581
    assert gather_call(L, n_dst=(1 << 24) + 1) == 583
    assert gather_call(L, n_group=1 << 13, n_src=1 << 12) == 583
    for p in ("parent", "src", "dst", "ws"):
        assert gather_call(L, **{p: None}) == 582
    assert gather_call(L, parent_len=7) == 582
    assert gather_call(L, src_bytes=239) == 582
    assert gather_call(L, dst_bytes=319) == 582
    assert gather_call(L, ws_bytes=255) == 582
    assert gather_call(L, ws=P + 64) == 591


def test_workspace_sizes(L):
    assert L.lossk_decode_workspace_bytes(L.KIND_BEAM_SELECT, 0, 1, 1, 1) == -1
    assert L.lossk_decode_workspace_bytes(L.KIND_BEAM_SELECT, 1, 65, 1, 1) == -1
    assert L.lossk_decode_workspace_bytes(99, 1, 1, 1, 1) == -1
    for kind, sizes in ((L.KIND_BEAM_SELECT, (3, 5, 777, 9)), (L.KIND_CACHE, (7, 100))):
        nb = L.lossk_decode_workspace_bytes(kind, *sizes)
        assert nb >= 256 and nb % 256 == 0
    with pytest.raises(ValueError):
        L.decode_workspace(L.KIND_BEAM_SELECT, 1, 1, 1, 1000)


def test_reference_orders_candidates():
    """The tests' own definition on a case worked by hand: two beams, ties to the lower beam and token."""
    import decode_ref as ref
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.25, 0.25, 0.5]]))
    r = ref.beam_select(x, np.array([[0.0, 0.0]]), 4)
    assert r["parent"].tolist() == [[0, 1, 0, 0]] and r["token"].tolist() == [[0, 2, 1, 2]]
    np.testing.assert_allclose(np.exp(r["score"]), [[0.5, 0.5, 0.25, 0.25]], rtol=1e-12)
    np.testing.assert_allclose(r["lse"], 0.0, atol=1e-12)
