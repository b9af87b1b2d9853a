"""Decoding calls on a stream that is not the current one, with workspace and outputs left to them: what the
current stream allocates and writes while they wait their turn must not be theirs."""
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


def on_a_busy_stream(call, sizes):
    """The call's result on a stream that is busy for some milliseconds, the current stream writing meanwhile."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    out = call(side)
    for _ in range(3):
        for n in sizes:
            torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    side.synchronize()
    torch.cuda.synchronize()
    return out


SIZES = [256, 512, 1 << 10, 1 << 12, 1 << 14, 1 << 16, 1 << 20, 1 << 22, 1 << 24, 1 << 26]


def test_selection_and_gather(L):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(32, 20011, device="cuda", generator=g)
    s = -torch.rand(8, 4, device="cuda", generator=g)
    want = L.lossk_beam_select(x, s, 6)
    got = on_a_busy_stream(lambda st: L.lossk_beam_select(x, s, 6, stream=st), SIZES)
    assert all(torch.equal(got[k], want[k]) for k in want)
    src = torch.randn(8, 4, 1001, device="cuda", generator=g)
    a = L.lossk_beam_gather(src, want["parent"])
    b = on_a_busy_stream(lambda st: L.lossk_beam_gather(src, want["parent"], stream=st), SIZES)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention(L, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(300, 16, 2, 64, device="cuda", generator=g).to(dtype) for _ in range(2))
    q = torch.randn(4, 8, 64, device="cuda", generator=g).to(dtype)
    table = torch.randperm(300, device="cuda", generator=g).int().view(4, 75)
    lens = torch.tensor([1200, 33, 700, 1], dtype=torch.int32, device="cuda")
    for share in (1, 2):
        want = L.lossk_paged_attn(q, k, v, table, lens, share=share)
        got = on_a_busy_stream(lambda st: L.lossk_paged_attn(q, k, v, table, lens, share=share, stream=st), SIZES)
        assert torch.equal(got, want)


def test_pages(L):
    g = torch.Generator(device="cuda").manual_seed(3)
    pool0 = torch.randn(2, 40, 4, 8, device="cuda", generator=g)
    table0 = torch.tensor([[3, 9, -1, -1], [7, -1, -1, -1]], dtype=torch.int32, device="cuda")
    lens0 = torch.tensor([6, 3], dtype=torch.int32, device="cuda")
    ref0 = torch.zeros(40, dtype=torch.int32, device="cuda")
    ref0[[3, 9, 7]] = 1
    parent = torch.tensor([[0, 0, 1]], dtype=torch.int32, device="cuda")

    def steps(st):
        pool, ref = pool0.clone(), ref0.clone()
        torch.cuda.synchronize()                       # (the calls alone are what the busy stream holds up)
        if st is not None:
            with torch.cuda.stream(st):
                torch.cuda._sleep(20_000_000)
        t, n = L.lossk_cache_fork(parent, table0, lens0, ref, 4, stream=st)
        L.lossk_cache_reserve(t, n, ref, pool, 4, stream=st)
        c, r, live = L.lossk_cache_compact(t, n, ref, pool, 4, stream=st)
        return t, n, ref, pool, c, r, live
    want = steps(None)
    got = on_a_busy_stream(steps, SIZES)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
