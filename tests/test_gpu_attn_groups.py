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
