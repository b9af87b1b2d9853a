"""The cache's pages on the GPU against a cache kept by hand: tables, counts and every byte of the pool."""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from conftest import build_lib
    build_lib()
    import output_projection_cross_gb300 as L
    assert torch.cuda.is_available()
    return L


class Pair:
    """The same cache on the GPU and by hand."""

    def __init__(self, L, rng, n_seq, n_pages, page, max_pages, planes=4, row=(2, 8), dtype=torch.bfloat16,
                 layout="token"):
        self.L, self.rng, self.page, self.max_pages, self.row = L, rng, page, max_pages, row
        shape = (planes, n_pages, page) + row
        data = torch.from_numpy(rng.integers(-100, 100, shape).astype(np.float32)).to(dtype)
        self.layout = layout
        self.pool = data.cuda()
        if layout == "head":
            self.pool = self.pool.transpose(2, 3).contiguous()
        self.hand = ref.Cache(data.float().numpy(), page, [[] for _ in range(n_seq)])
        self.table = torch.full((n_seq, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.ws = L.decode_workspace(L.KIND_CACHE, 4 * n_seq, n_pages)

    def same(self, status=580):
        assert self.L.lossk_device_status(self.ws) == status
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.hand.table(self.max_pages))
        np.testing.assert_array_equal(self.lens.cpu().numpy(), self.hand.lens)
        np.testing.assert_array_equal(self.ref.cpu().numpy(), self.hand.ref())
        pool = self.pool.transpose(2, 3) if self.layout == "head" else self.pool
        np.testing.assert_array_equal(pool.float().cpu().numpy(), self.hand.pool)

    def fork(self, parent):
        n_src = len(self.hand.rows) // len(parent)
        self.hand.fork(parent, n_src)
        par = torch.tensor(parent, dtype=torch.int32, device="cuda")
        self.table, self.lens = self.L.lossk_cache_fork(par, self.table, self.lens, self.ref, self.page, ws=self.ws)

    def add(self, n_new, scalar=False):
        """Reserves and writes n_new[i] tokens, then counts them; False where the pool has too few pages."""
        L = self.L
        before = self.ref.clone()
        ok = self.hand.reserve(n_new)
        arg = n_new[0] if scalar else torch.tensor(n_new, dtype=torch.int32, device="cuda")
        L.lossk_cache_reserve(self.table, self.lens, self.ref, self.pool, self.page, arg, ws=self.ws)
        if not ok:
            assert torch.equal(before, self.ref)
            self.same(584)
            return False
        first = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        n = int(first[-1])
        if n:
            kv = torch.from_numpy(self.rng.integers(-100, 100, (n, 2) + self.row).astype(np.float32)).to(self.pool.dtype)
            g = kv.cuda()
            pages = [self.pool[i].transpose(1, 2) if self.layout == "head" else self.pool[i] for i in (0, 1)]
            one = all(x == 1 for x in n_new)
            L.lossk_cache_write(g[:, 0], g[:, 1], pages[0], pages[1], self.table, self.lens,
                                first=None if one else torch.from_numpy(first).cuda(), ws=self.ws)
            self.hand.write(kv[:, 0].float().numpy(), kv[:, 1].float().numpy(), first)
        self.lens += torch.tensor(n_new, dtype=torch.int32, device="cuda")
        self.hand.lens = [a + b for a, b in zip(self.hand.lens, n_new)]
        return True

    def compact(self, in_place=False):
        n = self.hand.compact()
        self.table, self.ref, live = self.L.lossk_cache_compact(
            self.table, self.lens, self.ref, self.pool, self.page, ws=self.ws,
            table_out=self.table if in_place else None)
        assert live.item() == n


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("dtype,row", [(torch.bfloat16, (2, 8)), (torch.float32, (1, 4)), (torch.float16, (3, 24))])
@pytest.mark.parametrize("page", [1, 4, 16])
def test_a_search_kept_by_hand(L, page, dtype, row, layout):
    """Prompts of uneven length, then beams that fork, grow, are dropped and compacted, step by step."""
    rng = np.random.default_rng([page, row[0]])
    groups, beams = 3, 4
    p = Pair(L, rng, groups, 640 // page + 40, page, 200 // page + 2, row=row, dtype=dtype, layout=layout)
    assert p.add([5, 0, 33])
    p.same()
    p.fork([[0] * beams] * groups)                     # one row per prompt becomes one per beam
    p.same()
    for step in range(12):
        assert p.add([1] * (groups * beams), scalar=step % 2 == 0)
        p.same()
        parent = rng.integers(0, beams, (groups, beams)).tolist()
        if step % 4 == 3:
            parent[step % 3][1] = -1
        p.fork(parent)
        p.same()
        if step % 5 == 4:
            p.compact(in_place=step == 4)
            p.same()
        if step == 8:
            drop = [1 if i % 5 == 0 else 0 for i in range(groups * beams)]
            p.hand.free(drop)
            L.lossk_cache_free(p.table, p.lens, p.ref, page, torch.tensor(drop, dtype=torch.uint8, device="cuda"),
                               ws=p.ws)
            p.same()
    p.hand.free([1] * (groups * beams))
    L.lossk_cache_free(p.table, p.lens, p.ref, page, ws=p.ws)
    p.same()
    assert int(p.ref.abs().sum()) == 0


def test_many_sequences(L):
    """More sequences than the planning block has threads, more pages than it scans at once."""
    rng = np.random.default_rng(3)
    groups, beams = 700, 3
    p = Pair(L, rng, groups, 9000, 8, 6, planes=2, row=(1, 8))
    assert p.add(rng.integers(0, 20, groups).tolist())
    p.fork([[0] * beams] * groups)
    assert p.add([1] * (groups * beams))
    p.same()
    p.fork(rng.integers(-1, beams, (groups, beams)).tolist())
    assert p.add(rng.integers(0, 9, groups * beams).tolist())
    p.same()
    p.compact()
    p.same()


def test_a_page_shared_beyond_the_call_is_left_alone(L):
    """Two of three sharers ask for room: both get copies, for the third still holds the page."""
    rng = np.random.default_rng(4)
    p = Pair(L, rng, 1, 20, 4, 5)
    assert p.add([6])
    p.fork([[0, 0, 0]])
    assert p.add([1, 0, 1])
    p.same()
    assert p.hand.rows[1][1] not in (p.hand.rows[0][1], p.hand.rows[2][1])


def test_too_few_pages_change_nothing(L):
    rng = np.random.default_rng(5)
    p = Pair(L, rng, 2, 6, 4, 8)
    assert p.add([9, 4])
    p.same()
    p.fork([[0, 0, 1, 1]])
    assert not p.add([1, 1, 5, 4])
    assert p.add([1, 0, 1, 0])
    p.same()


@pytest.mark.parametrize("what", ["entries", "long", "negative", "page", "new"])
def test_reserve_refuses_as_a_whole(L, what):
    rng = np.random.default_rng(6)
    p = Pair(L, rng, 3, 30, 4, 4)
    assert p.add([6, 3, 16])
    t, n, r, pool = p.table.clone(), p.lens.clone(), p.ref.clone(), p.pool.clone()
    n_new = torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda")
    status = 586
    if what == "entries":
        n_new[2], status = 1, 584                      # 17 tokens do not fit in four pages
    elif what == "long":
        p.lens[0] = 17
    elif what == "negative":
        p.lens[1] = -1
    elif what == "page":
        p.table[0, 1] = 30
    elif what == "new":
        n_new[0] = -2
    t, n = p.table.clone(), p.lens.clone()
    L.lossk_cache_reserve(p.table, p.lens, p.ref, p.pool, 4, n_new, ws=p.ws)
    assert L.lossk_device_status(p.ws) == status
    assert torch.equal(t, p.table) and torch.equal(r, p.ref) and torch.equal(pool, p.pool)
    assert L.lossk_device_status(p.ws) == 580


def test_fork_reports_what_is_out_of_range(L):
    rng = np.random.default_rng(7)
    for what in ("parent", "low", "page", "len"):
        p = Pair(L, rng, 2, 30, 4, 4)
        assert p.add([6, 9])
        par = [[0, 1, 1]]
        if what == "parent":
            par = [[0, 2, 1]]
        elif what == "low":
            par = [[0, -2, 1]]
        elif what == "page":
            p.table[1, 1] = -7
        else:
            p.lens[1] = 17
        t, n = L.lossk_cache_fork(torch.tensor(par, dtype=torch.int32, device="cuda"), p.table, p.lens, p.ref, 4,
                                  ws=p.ws)
        assert L.lossk_device_status(p.ws) == 586
        assert n[0].item() == 6 and t[0].tolist() == p.hand.table(4)[0].tolist()
        if what in ("parent", "low"):
            assert n.tolist() == [6, 0, 9] and t[1].tolist() == [-1] * 4
        elif what == "page":
            assert t[1, 1].item() == -1 and t[1, 0].item() == p.hand.rows[1][0]
        else:
            assert n.tolist() == [6, 0, 0]


def test_compact_reports_a_page_that_is_free(L):
    rng = np.random.default_rng(8)
    p = Pair(L, rng, 2, 30, 4, 4)
    assert p.add([6, 9])
    free = p.table[0, 0].item()
    p.ref[free] = 0
    p.table[1, 0] = 30
    t, r, n = L.lossk_cache_compact(p.table, p.lens, p.ref, p.pool, 4, ws=p.ws)
    assert L.lossk_device_status(p.ws) == 586
    assert n.item() == 4 and t[0, 0].item() == -1 and t[1, 0].item() == -1


def test_copy(L):
    rng = np.random.default_rng(9)
    ws = L.decode_workspace(L.KIND_CACHE, 1, 50)
    for shape, dtype in (((3, 50, 4, 4), torch.float32), ((1, 50, 16, 8, 128), torch.bfloat16), ((2, 50, 16), torch.uint8)):
        pool = torch.from_numpy(rng.integers(0, 100, shape)).cuda().to(dtype)
        want = pool.clone()
        ids = rng.permutation(50)
        src, dst = ids[:20], ids[20:40]
        want[:, torch.from_numpy(dst).cuda()] = want[:, torch.from_numpy(src).cuda()]
        src, dst = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (src, dst))
        src, dst = torch.cat([src, src.new_tensor([-1])]), torch.cat([dst, dst.new_tensor([-1])])
        L.lossk_cache_copy(src, dst, pool, ws=ws)
        assert L.lossk_device_status(ws) == 580
        assert torch.equal(pool, want)
        for a, b in ((50, 1), (1, 50), (-1, 3), (3, -5)):
            L.lossk_cache_copy(src.new_tensor([a]), src.new_tensor([b]), pool, ws=ws)
            assert L.lossk_device_status(ws) == 586
            assert torch.equal(pool, want)


def test_a_pool_whose_planes_and_pages_lie_apart(L):
    """Strides between planes and pages that are larger than a page."""
    big = torch.arange(2 * 12 * 40, device="cuda", dtype=torch.float32).view(2, 12, 40)
    pool = big[:, 1:11, :16]
    want = big.clone()
    want[:, 4, :16] = want[:, 2, :16]
    L.lossk_cache_copy(torch.tensor([1], dtype=torch.int32, device="cuda"),
                       torch.tensor([3], dtype=torch.int32, device="cuda"), big[:, 1:11, :16][:, :, :16])
    # (the first page of the view starts 160 bytes in: a multiple of 16)
    torch.cuda.synchronize()
    assert torch.equal(big, want) and torch.equal(pool, want[:, 1:11, :16])


@pytest.mark.parametrize("hd", [1, 3, 8, 100])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_write_odd_rows_and_strided_input(L, hd, dtype):
    """Head sizes that allow no wide word, rows that are slices of a wider projection."""
    rng = np.random.default_rng(hd)
    kv, page, n = 3, 5, 7
    pool = torch.zeros((2, 20, page, kv, hd), device="cuda", dtype=dtype)
    table = torch.arange(14, dtype=torch.int32, device="cuda").view(7, 2)
    lens = torch.tensor([0, 1, 4, 5, 6, 8, 9], dtype=torch.int32, device="cuda")
    wide = torch.randn((n, 2 * kv * hd + 5), device="cuda").to(dtype)
    k, v = wide[:, 5:5 + kv * hd].unflatten(1, (kv, hd)), wide[:, 5 + kv * hd:].unflatten(1, (kv, hd))
    ws = L.decode_workspace(L.KIND_CACHE, n, 20)
    L.lossk_cache_write(k, v, pool[0], pool[1], table, lens, ws=ws)
    assert L.lossk_device_status(ws) == 580
    want = torch.zeros_like(pool)
    for i, m in enumerate(lens.tolist()):
        want[0, table[i, m // page], m % page] = k[i]
        want[1, table[i, m // page], m % page] = v[i]
    assert torch.equal(pool, want)
    # no room: one token past the table, one on an entry without a page
    lens[3], table[4, 1] = 10, -1
    before = pool.clone()
    L.lossk_cache_write(k, v, pool[0], pool[1], table, lens, ws=ws)
    assert L.lossk_device_status(ws) == 586
    assert torch.equal(pool[:, 6:10], before[:, 6:10])


def test_offsets_beyond_32_bits(L):
    """A pool of over 4 GiB a plane: pages, rows and copies at its far end."""
    n_pages, page = 1100, 64
    pool = torch.empty((2, n_pages, page, 128, 256), device="cuda", dtype=torch.bfloat16)
    pool[:, n_pages - 3:] = 0
    assert pool[0].numel() * 2 > 1 << 32
    ws = L.decode_workspace(L.KIND_CACHE, 1, n_pages)
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([63], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((1, 128, 256), device="cuda").bfloat16() for _ in range(2))
    L.lossk_cache_write(k, v, pool[0], pool[1], table, lens, ws=ws)
    L.lossk_cache_copy(table[0], table[0] - 1, pool, ws=ws)
    assert L.lossk_device_status(ws) == 580
    for p in (n_pages - 1, n_pages - 2):
        assert torch.equal(pool[0, p, 63], k[0]) and torch.equal(pool[1, p, 63], v[0])
    assert pool[:, n_pages - 3].abs().sum() == 0
    ref_ = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    ref_[n_pages - 1] = 1
    t, r, n = L.lossk_cache_compact(table, lens, ref_, pool, page, ws=ws)
    assert n.item() == 1 and t.item() == 0 and r[0].item() == 1 and r.sum().item() == 1
    assert torch.equal(pool[:, 0], pool[:, n_pages - 1])


def test_pages_in_a_graph_and_on_another_stream(L):
    rng = np.random.default_rng(10)
    p = Pair(L, rng, 4, 60, 4, 8)
    assert p.add([6, 3, 9, 4])
    par = torch.tensor([[0, 0, 2, 3]], dtype=torch.int32, device="cuda")
    out, n_out, ref0 = torch.empty_like(p.table), torch.empty_like(p.lens), p.ref.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        p.ref.copy_(ref0)
        L.lossk_cache_fork(par, p.table, p.lens, p.ref, 4, table_out=out, lens_out=n_out, ws=p.ws)
        L.lossk_cache_reserve(out, n_out, p.ref, p.pool, 4, ws=p.ws)
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    p.hand.fork(par.tolist(), 4)
    assert p.hand.reserve([1] * 4)
    for _ in range(2):
        out.fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out.cpu().numpy(), p.hand.table(8))
        np.testing.assert_array_equal(p.ref.cpu().numpy(), p.hand.ref())
        np.testing.assert_array_equal(p.pool.float().cpu().numpy(), p.hand.pool)
