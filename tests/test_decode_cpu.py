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


# ---- the cache's pages ---------------------------------------------------------------

def call(fn, a, over):
    assert not set(over) - set(a), set(over) - set(a)
    a.update(over)
    return fn(*a.values())


def fork_call(L, **over):
    return call(L.lib.lossk_cache_fork, dict(
        n_group=2, n_src=3, n_dst=4, max_pages=5, page=16, n_pages=40, parent=P, parent_len=8, table=P, table_len=30,
        table_stride=5, lens=P, lens_len=6, ref=P, ref_len=40, table_out=2 * P, out_len=40, out_stride=5,
        lens_out=2 * P, lens_out_len=8, ws=P, ws_bytes=256, stream=None), over)


def reserve_call(L, **over):
    return call(L.lib.lossk_cache_reserve, dict(
        n_seq=6, max_pages=5, page=16, n_pages=40, n_new_all=1, n_new=None, n_new_len=0, table=P, table_len=30,
        table_stride=5, lens=P, lens_len=6, ref=P, ref_len=40, pool=P, pool_bytes=2 * 40 * 512, n_planes=2,
        plane_stride=40 * 512, page_stride=512, page_bytes=512, ws=P, ws_bytes=1 << 20, stream=None), over)


def free_call(L, **over):
    return call(L.lib.lossk_cache_free, dict(
        n_seq=6, max_pages=5, page=16, n_pages=40, drop=P, drop_len=6, table=P, table_len=30, table_stride=5, lens=P,
        lens_len=6, ref=P, ref_len=40, ws=P, ws_bytes=256, stream=None), over)


def compact_call(L, **over):
    return call(L.lib.lossk_cache_compact, dict(
        n_seq=6, max_pages=5, page=16, n_pages=40, table=P, table_len=30, table_stride=5, lens=P, lens_len=6, ref=P,
        ref_len=40, table_out=2 * P, out_len=30, out_stride=5, ref_out=2 * P, ref_out_len=40, n_live=P, pool=P,
        pool_bytes=2 * 40 * 512, n_planes=2, plane_stride=40 * 512, page_stride=512, page_bytes=512, ws=P,
        ws_bytes=1 << 20, stream=None), over)


def copy_call(L, **over):
    return call(L.lib.lossk_cache_copy, dict(
        n_copy=3, n_pages=40, src=P, src_len=3, dst=P, dst_len=3, pool=P, pool_bytes=2 * 40 * 512, n_planes=2,
        plane_stride=40 * 512, page_stride=512, page_bytes=512, ws=P, ws_bytes=256, stream=None), over)


def write_call(L, **over):
    return call(L.lib.lossk_cache_write, dict(
        n_tok=6, n_seq=6, n_kv=2, hd=8, max_pages=5, page=16, n_pages=40, dtype=1, k_new=P, v_new=P, new_len=96,
        new_stride=16, k=P, v=P, pages_len=40 * 256, page_stride=256, tok_stride=16, head_stride=8, table=P,
        table_len=30, table_stride=5, lens=P, lens_len=6, first=None, first_len=0, ws=P, ws_bytes=256, stream=None),
        over)


@pytest.mark.parametrize("fn,sizes", [
    (fork_call, ("n_group", "n_src", "n_dst", "max_pages", "page", "n_pages")),
    (reserve_call, ("n_seq", "max_pages", "page", "n_pages", "n_planes", "page_bytes")),
    (free_call, ("n_seq", "max_pages", "page", "n_pages")),
    (compact_call, ("n_seq", "max_pages", "page", "n_pages", "n_planes", "page_bytes")),
    (copy_call, ("n_copy", "n_pages", "n_planes", "page_bytes")),
    (write_call, ("n_tok", "n_seq", "n_kv", "hd", "max_pages", "page", "n_pages"))])
def test_cache_sizes_refused(L, fn, sizes):
    for s in sizes:
        assert fn(L, **{s: 0}) == 581, s
        if s != "page_bytes":
            assert fn(L, **{s: (1 << 24) + 1}) == 583, s


@pytest.mark.parametrize("fn,pointers,shorts", [
    (fork_call, ("parent", "table", "lens", "ref", "table_out", "lens_out", "ws"),
     dict(parent_len=7, table_len=29, table_stride=4, lens_len=5, ref_len=39, out_len=39, out_stride=4,
          lens_out_len=7, ws_bytes=255, table_out=P, lens_out=P)),
    (reserve_call, ("table", "lens", "ref", "pool", "ws"),
     dict(table_len=29, table_stride=4, lens_len=5, ref_len=39, pool_bytes=2 * 40 * 512 - 1, page_stride=496,
          plane_stride=-16, n_new_all=-1, ws_bytes=512)),
    (free_call, ("table", "lens", "ref", "ws"),
     dict(drop_len=5, table_len=29, table_stride=4, lens_len=5, ref_len=39, ws_bytes=255)),
    (compact_call, ("table", "lens", "ref", "table_out", "ref_out", "n_live", "pool", "ws"),
     dict(table_len=29, lens_len=5, ref_len=39, out_len=29, out_stride=4, ref_out_len=39, ref_out=P,
          pool_bytes=2 * 40 * 512 - 1, page_stride=496, ws_bytes=512)),
    (copy_call, ("src", "dst", "pool", "ws"),
     dict(src_len=2, dst_len=2, pool_bytes=2 * 40 * 512 - 1, page_stride=496, ws_bytes=255)),
    (write_call, ("k_new", "v_new", "k", "v", "table", "lens", "ws"),
     dict(dtype=9, new_len=95, new_stride=15, pages_len=40 * 256 - 1, page_stride=-1, tok_stride=17, head_stride=9,
          table_len=29, lens_len=5, n_tok=5, ws_bytes=255))])
def test_cache_arguments_refused(L, fn, pointers, shorts):
    for p in pointers:
        assert fn(L, **{p: None}) == 582, p
    for k, v in shorts.items():
        assert fn(L, **{k: v}) == 582, k
    assert fn(L, ws=P + 128) == 591


def test_cache_alignment_refused(L):
    for fn in (reserve_call, compact_call, copy_call):
        assert fn(L, pool=P + 8, pool_bytes=1 << 20) == 591
        assert fn(L, page_bytes=504) == 591
        assert fn(L, page_stride=520, pool_bytes=1 << 20) == 591
    assert write_call(L, k=P + 1) == 591
    assert write_call(L, dtype=0, k_new=P + 2) == 591
    assert write_call(L, first=P, first_len=6) == 582
    assert fork_call(L, ref=P + 2) == 591


def test_reference_cache_by_hand():
    """Two beams fork from one sequence of three tokens in pages of two: the shared half-full page is
    copied for the first and kept by the second."""
    import decode_ref as ref
    c = ref.Cache(np.arange(12.0).reshape(2, 6, 1, 1).repeat(2, 2), 2, [[4, 1]])
    c.lens = [3]
    c.fork([[0, 0]], 1)
    assert c.ref().tolist() == [0, 2, 0, 0, 2, 0]
    assert c.reserve([1, 1])
    assert c.rows == [[4, 0], [4, 1]] and c.ref().tolist() == [1, 1, 0, 0, 2, 0]
    assert (c.pool[:, 0] == c.pool[:, 1]).all()
    c.lens = [4, 4]
    assert not c.reserve([1, 5]) and c.reserve([1, 0]) and c.rows[0] == [4, 0, 2]
    c.free([1, 0])
    assert c.compact() == 2 and c.rows == [[], [0, 1]]


# ---- attention of one new token ---------------------------------------------------------

def attn_call(L, **over):
    return call(L.lib.lossk_paged_attn, dict(
        n_seq=6, n_q=8, n_kv=2, hd=64, max_pages=5, page=16, n_pages=40, share=1, dtype=1, q=P, q_len=6 * 512,
        q_stride=512, k=P, v=P, pages_len=40 * 2048, page_stride=2048, tok_stride=128, head_stride=64, table=P,
        table_len=30, table_stride=5, lens=P, lens_len=6, max_len=0, window=0, scale=0.125, out=P, out_len=6 * 512,
        lse=P, ws=P, ws_bytes=1 << 28, stream=None), over)


def test_attention_refusals(L):
    for size in ("n_seq", "n_q", "n_kv", "hd", "max_pages", "page", "n_pages", "share"):
        assert attn_call(L, **{size: 0}) == 581, size
    for size in ("n_seq", "n_q", "max_pages", "page", "n_pages"):
        assert attn_call(L, **{size: (1 << 24) + 1}) == 583, size
    assert attn_call(L, hd=264) == 583
    assert attn_call(L, max_pages=1 << 20, page=1 << 11) == 583
    for p in ("q", "k", "v", "table", "lens", "out", "ws"):
        assert attn_call(L, **{p: None}) == 582, p
    for k, v in dict(n_q=7, share=4, q_len=6 * 512 - 1, q_stride=511, pages_len=40 * 2048 - 1, table_len=29,
                     table_stride=4, lens_len=5, out_len=6 * 512 - 1, max_len=-1, window=-1, dtype=5,
                     page_stride=-8, tok_stride=136,
                     ws_bytes=L.lossk_decode_workspace_bytes(L.KIND_PAGED_ATTN, 6, 8, 2, 64) - 1).items():
        assert attn_call(L, **{k: v}) == 582, k
    for p in ("q", "k", "v", "out"):
        assert attn_call(L, **{p: P + 8}) == 591, p
    assert attn_call(L, ws=P + 128) == 591
    assert attn_call(L, hd=60, q_len=1 << 20) == 591
    assert attn_call(L, tok_stride=132, pages_len=1 << 20) == 591
    assert attn_call(L, q_stride=516, q_len=1 << 20) == 591
    for x in (float("nan"), float("inf"), 1e300):
        assert attn_call(L, scale=x) == 585
    assert attn_call(L, scale=float("nan"), ws=P + 1) == 591
    assert L.lossk_decode_workspace_bytes(L.KIND_PAGED_ATTN, 1, 1, 1, 257) == -1


def test_reference_attention_by_hand():
    import decode_ref as ref
    k = np.zeros((2, 2, 1, 1))
    k[1, :, 0, 0] = [0.0, math_log3 := float(np.log(3.0))]
    v = np.zeros((2, 2, 1, 1))
    v[1, :, 0, 0] = [4.0, 8.0]
    o, lse = ref.attend(np.ones((1, 1, 1)), k, v, np.array([[1]]), [2], 2, 1.0)
    np.testing.assert_allclose([o.item(), lse.item()], [7.0, np.log(4.0)], rtol=1e-12)
    o, lse = ref.attend(np.ones((1, 1, 1)), k, v, np.array([[1]]), [2], 2, 1.0, window=1)
    np.testing.assert_allclose([o.item(), lse.item()], [8.0, math_log3], rtol=1e-12)
