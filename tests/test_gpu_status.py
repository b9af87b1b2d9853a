"""lossk_device_status on workspaces of the losses' calls, which clear no more of the header than they use."""
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


@pytest.mark.parametrize("byte", [0x7F, 0xFF, 1])
def test_what_memory_held_is_no_status(L, byte):
    ws = torch.full((1 << 20,), byte, dtype=torch.uint8, device="cuda")
    ws[:16] = 0                                        # the error word and what each call counts
    y = torch.zeros(64, dtype=torch.int64, device="cuda")
    assert L.lossk_targets_check(y, 10, ws=ws) == 580
    before = ws.clone()
    assert L.lossk_device_status(ws) == 580
    assert torch.equal(ws, before)
    assert L.lossk_selftest_wait(4, 2, 5_000_000, ws)[0] == 590
    assert L.lossk_device_status(ws) == 590
    assert L.lossk_device_status(ws) == 580


def test_a_decoding_call_s_fault_beside_an_error(L):
    """Both are cleared; the error is what is reported, as of the two it is the larger code."""
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    src, bad = torch.ones(1, 2, 4, device="cuda"), torch.tensor([[7]], dtype=torch.int32, device="cuda")
    L.lossk_beam_gather(src, bad, ws=ws)
    assert L.lossk_selftest_wait(4, 2, 5_000_000, ws)[0] == 590
    assert L.lossk_device_status(ws) == 590 and L.lossk_device_status(ws) == 580
    L.lossk_beam_gather(src, bad, ws=ws)
    assert L.lossk_device_status(ws) == 586 and L.lossk_device_status(ws) == 580
