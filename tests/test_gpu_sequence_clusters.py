"""The policy loss from given logits where a cluster of blocks takes a row: two, four and eight blocks, rows that count
among rows that do not, refused calls between, all on one workspace."""
import pytest
import torch

import output_projection_cross_gb300 as L
from test_gpu_sequence import CODE, Case, check_policy, run_policy
from test_gpu_sequence_edges import same

pytestmark = pytest.mark.gpu

# rows of 90, 200 and 600 KB that are more than the GPU has places for, then few rows in as many pieces as there are
WIDE = [dict(n=500, V=45001, dtype="bf16"), dict(n=301, V=50003, dtype="f32"), dict(n=200, V=300001, dtype="f16"),
        dict(n=90, V=32003, dtype="bf16"), dict(n=48, V=32000, dtype="f16"), dict(n=7, V=20011, dtype="f32")]


@pytest.mark.parametrize("kw", WIDE, ids=str)
@pytest.mark.parametrize("masked", [0.0, 0.5, 0.95])
def test_rows_of_a_cluster(kw, masked):
    c = Case(masked=masked, **kw)
    ws = L.sequence_workspace(1, c.n, 1, c.V, 0, CODE[c.dtype])
    out = run_policy(c, kl=0.1, ws=ws)
    check_policy(c, out, kl=0.1)
    for _ in range(5):
        same(out, run_policy(c, kl=0.1, ws=ws))
    assert L.lossk_device_status(ws) == 580


@pytest.mark.parametrize("kw", WIDE, ids=str)
def test_a_refused_call_between(kw):
    c = Case(masked=0.3, **kw)
    ws = L.sequence_workspace(1, c.n, 1, c.V, 0, CODE[c.dtype])
    want = run_policy(c, ws=ws)
    wrong = c.targets.clone()
    wrong[torch.nonzero(c.on)[0]] = c.V
    c.targets, good = wrong, c.targets
    marked = torch.full_like(c.logits, 7.0)
    for _ in range(3):
        run_policy(c, ws=ws, grad_logits=marked)
        assert L.lossk_device_status(ws) == 586
    assert (marked == 7.0).all()
    c.targets = good
    same(want, run_policy(c, ws=ws))
    assert L.lossk_device_status(ws) == 580
