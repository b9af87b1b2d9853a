"""What the losses of sequences leave in a workspace's header, and what later calls make of it."""
import pytest
import torch

import output_projection_cross_gb300 as L
from test_gpu_sequence import CODE, Case, check_policy, check_preference, run_policy, run_preference
from test_gpu_sequence_edges import HEADS, ROWS, of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", HEADS + ROWS, ids=str)
@pytest.mark.parametrize("what", ["target", "first"])
def test_calls_idle_until_the_status_is_read(kw, what):
    """A refused call, then good ones on the same workspace: they write nothing before the status has been read."""
    c = Case(seqs=4, **kw)
    good = c.targets.clone(), c.first.clone()
    ws = L.sequence_workspace(0 if c.d else 1, c.n, max(c.d, 1), c.V, 4, CODE[c.dtype])
    mark = lambda *shape: torch.full(shape, 7.0, device="cuda")  # noqa: E731
    outs = dict(scalars_out=mark(4), logp_out=mark(c.n))
    grads = dict(d_hidden=mark(c.n, c.d), d_weight=mark(c.V, c.d)) if c.d else dict(grad_logits=torch.full_like(c.logits, 7.0))
    outs.update(grads)
    policy, pair = dict(per_token_out=mark(c.n)), dict(per_pair_out=mark(2), log_ratio_out=mark(4))
    if what == "target":
        c.targets[c.n // 2] = c.V
    else:
        c.first[4] = c.n + 1
    run_policy(c, ws=ws, **outs, **policy)
    c.targets, c.first = good
    for flags in (0, L.SEQ_RATIO, L.ACCUMULATE_GRADS):
        run_policy(c, flags, ws=ws, **outs, **policy)
    run_preference(c, ws=ws, **outs, **pair)
    torch.cuda.synchronize()
    for t in (*outs.values(), *policy.values(), *pair.values()):
        assert (t == 7.0).all()
    assert L.lossk_device_status(ws) == 586 and L.lossk_device_status(ws) == 580
    check_policy(c, run_policy(c, ws=ws, **of(c)))
    check_preference(c, run_preference(c, ws=ws, **of(c)))
    assert L.lossk_device_status(ws) == 580


def test_what_is_no_status_is_none():
    """A word that no call leaves there stops nothing and hides nothing."""
    c = Case(seqs=4, **HEADS[0])
    ws = L.sequence_workspace(0, c.n, c.d, c.V, 4, CODE[c.dtype])
    words, good = ws[:256].view(torch.int32), c.targets.clone()
    for word in (1, 583, 587, -1):
        words[5] = word
        check_policy(c, run_policy(c, ws=ws, **of(c)))
        assert L.lossk_device_status(ws) == 580
        c.targets[3] = -1
        run_policy(c, ws=ws, **of(c))
        assert L.lossk_device_status(ws) == 586
        c.targets.copy_(good)
