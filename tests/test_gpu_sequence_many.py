"""The policy loss with far more sequences than tokens: what empty ones cost, and that they change nothing."""
import time

import pytest
import torch

import output_projection_cross_gb300 as L
from test_gpu_sequence import CODE, Case, check_policy, gen, run_policy

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(n=64, V=100, d=8, dtype="f32"), dict(n=64, V=300, d=64, dtype="bf16"), dict(n=64, V=900, dtype="f16"),
                                dict(n=8, V=500003, dtype="bf16")], ids=str)
@pytest.mark.parametrize("log2_seqs,limit", [(12, None), (20, None), (25, 0.45)])
def test_empty_sequences_between_tokens(kw, log2_seqs, limit):
    """Tokens scattered over up to 2^25 sequences, all but a few of them empty.  With the most of them a call is bound by the
    passes over their starts, 0.02 s; a walk from a token's sequence to the next token's took 1.3."""
    c = Case(**kw)
    S = 1 << log2_seqs
    at = torch.sort(torch.randint(0, S, (c.n,), device="cuda", generator=gen(2))).values
    at[0], at[-1] = 0, S - 1
    # first[s]: tokens of sequences before s
    first = torch.searchsorted(at, torch.arange(S + 1, device="cuda")).to(torch.int32)
    adv = torch.zeros(S, device="cuda")
    adv[at] = torch.randn(c.n, device="cuda", generator=gen(3))
    # the definition on the sequences that have a token
    own, index = torch.unique(at, return_inverse=True)
    c.first = torch.cat([torch.searchsorted(at, own), torch.tensor([c.n], device="cuda")]).to(torch.int32)
    few, c.first = c.first, first
    flags = L.SEQ_MEAN | L.SEQ_ADVANTAGES
    ws = L.sequence_workspace(0 if c.d else 1, c.n, max(c.d, 1), c.V, S, CODE[c.dtype])
    c.seq_adv = adv
    run_policy(c, flags, kl=0.1, ws=ws)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    out = run_policy(c, flags, kl=0.1, ws=ws)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    print("seconds", took)
    c.first, c.seq_adv = few, adv[own]
    check_policy(c, out, flags, kl=0.1, **({"grad": "float"} if c.d else {}))
    assert limit is None or took < limit
    assert L.lossk_device_status(ws) == 580
