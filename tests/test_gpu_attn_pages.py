"""Attention over a paged cache: every id that is no page is reported, whatever its value."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("share", [1, 2])
@pytest.mark.parametrize("bad", [-1, -2, -3, -(1 << 31), 12, (1 << 31) - 1])
def test_an_id_that_is_no_page(L, dtype, share, bad):
    rng = np.random.default_rng(1)
    k, v = (torch.from_numpy(rng.standard_normal((12, 16, 2, 64))).cuda().to(dtype) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((2, 4, 64))).cuda().to(dtype)
    table = np.array([[4, 7, 1, 0], [4, 7, 2, 3]], np.int32)
    lens = [60, 62]
    for row, col in ((0, 1), (1, 0), (0, 3), (1, 3)):
        t = table.copy()
        t[row, col] = bad
        ws = L.decode_workspace(L.KIND_PAGED_ATTN, 2, 4, 2, 64)
        out = L.lossk_paged_attn(q, k, v, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 share=share, ws=ws)
        assert L.lossk_device_status(ws) == 586
        # its tokens are left out: the other pages' alone, the last one's length unless that is the page
        kept = np.delete(table[row:row + 1], col, 1)
        n = 48 if col == 3 else lens[row] - 16
        args = (x.double().cpu().numpy() for x in (q[row:row + 1], k, v))
        r, _ = ref.attend(*args, kept, [n], 16, 0.125)
        eps = torch.finfo(dtype).eps
        # (half a step of the type, and 5e-5 for fp32 sums of values up to 4)
        assert (np.abs(out[row].double().cpu().numpy() - r[0]) <= eps / 2 * np.abs(r[0]) + 5e-5).all()
