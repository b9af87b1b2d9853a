"""The decoding calls begin while the kernel ahead of them in the stream ends: what that kernel
writes has to be read, and what it still reads must not be overwritten."""
import pytest
import torch

import output_projection_cross_gb300 as L

pytestmark = pytest.mark.gpu


def slow_copy(dst, src):
    """Writes dst late: each element depends on a long chain, several kernels deep."""
    x = src
    for _ in range(3):
        x = torch.cumsum(x.to(torch.float64).flatten(), 0).diff(prepend=torch.zeros(1, dtype=torch.float64, device=x.device))
        x = x.round().reshape(src.shape)
    torch.add(x.to(dst.dtype), 0, out=dst)


def test_select_reads_what_is_just_written():
    B, K, V = 3, 4, 20011
    g = torch.Generator(device="cuda").manual_seed(1)
    ws = L.decode_workspace(L.KIND_BEAM_SELECT, B, K, V, 6)
    out = L.beam_buffers(B, 6)
    scores = torch.zeros(B, K, device="cuda")
    logits = torch.zeros(B * K, V, device="cuda")
    kept, want = [], []
    inputs = [torch.randint(-1000, 1000, (B * K, V), device="cuda", generator=g).float() for _ in range(8)]
    for x in inputs:
        want.append(L.lossk_beam_select(x / 64, scores, 6)["token"].clone())
    torch.cuda.synchronize()
    for x in inputs:
        slow_copy(logits, x)
        logits.div_(64)
        L.lossk_beam_select(logits, scores, 6, out=out, ws=ws)
        kept.append(out["token"].clone())          # read while the next call is already queued
    torch.cuda.synchronize()
    for a, b in zip(kept, want):
        assert torch.equal(a, b)


def test_cache_and_attention_in_a_row():
    n, hq, hkv, hd, page, pages = 3, 8, 4, 64, 16, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    pool = torch.randn(2, pages, page, hkv, hd, device="cuda", generator=g).to(torch.bfloat16)
    table0 = torch.full((n, 8), -1, dtype=torch.int32, device="cuda")
    table0[:, :4] = torch.arange(4 * n, dtype=torch.int32, device="cuda").view(n, 4)
    lens0 = torch.tensor([60, 33, 47], dtype=torch.int32, device="cuda")
    ref0 = torch.zeros(pages, dtype=torch.int32, device="cuda")
    used = (lens0 + page - 1) // page
    for i in range(n):
        ref0[table0[i, :used[i]].long()] = 1
    parents = [torch.tensor([p], dtype=torch.int32, device="cuda") for p in ([0, 0, 2], [1, 2, 0], [2, 2, 2], [0, 1, 2])]
    ws, wa = L.decode_workspace(L.KIND_CACHE, n, pages), L.decode_workspace(L.KIND_PAGED_ATTN, n, hq, hkv, hd)
    q = torch.randn(n, hq, hd, device="cuda", generator=g).to(torch.bfloat16)
    news = [torch.randn(2, n, hkv, hd, device="cuda", generator=g).to(torch.bfloat16) for _ in parents]

    def steps(sync):
        kv, table, lens, ref = pool.clone(), table0.clone(), lens0.clone(), ref0.clone()
        t2, l2, out = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(q)
        parent = torch.empty_like(parents[0])
        got = []

        def step(*_):
            if sync:
                torch.cuda.synchronize()
        for p, new in zip(parents, news):
            slow_copy(parent, p)
            step()
            L.lossk_cache_fork(parent, table, lens, ref, page, table_out=t2, lens_out=l2, ws=ws)
            step()
            L.lossk_cache_reserve(t2, l2, ref, kv, page, ws=ws)
            step()
            L.lossk_cache_write(new[0], new[1], kv[0], kv[1], t2, l2, ws=ws)
            step()
            l2.add_(1)
            step()
            L.lossk_paged_attn(q, kv[0], kv[1], t2, l2, share=n, out=out, ws=wa)
            step()
            got.append((out.clone(), t2.clone(), l2.clone(), ref.clone()))
            step()
            table, t2, lens, l2 = t2, table, l2, lens
        torch.cuda.synchronize()
        assert L.lossk_device_status(ws) == 580 and L.lossk_device_status(wa) == 580
        return got

    want = steps(True)
    for _ in range(5):
        for a, b in zip(steps(False), want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
