"""The decoding calls together, as examples/beam_decode.py uses them: every hypothesis's score is the
sum of its tokens' log-probabilities under a plain forward pass without cache, pages or beams."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from conftest import build_lib
    build_lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import beam_decode
    return beam_decode


@pytest.mark.parametrize("page,alpha", [(16, 0.0), (4, 0.6)])
def test_scores_are_those_of_a_plain_forward_pass(ex, page, alpha):
    m = ex.Decoder(vocab=203, d=64, layers=2, q_heads=4, kv_heads=2, head_dim=32, seed=3)
    prompts = torch.randint(0, 203, (3, 9), generator=torch.Generator().manual_seed(4)).cuda()
    search = ex.BeamSearch(m, prompts, 3, 12, end_token=7, page=page, length_alpha=alpha)
    tokens, length, score = search.run(12)
    assert int(search.ref.abs().sum()) == 0                 # every page came back
    rank = score / length.clamp(min=1) ** alpha
    assert (rank[:, :-1] >= rank[:, 1:] - 1e-5).all()
    for b in range(3):
        seen = set()
        for k in range(3):
            n = int(length[b, k])
            seq = tokens[b, k, :n]
            assert (tokens[b, k, n:] == 7).all() and (n == 12 or seq[-1] == 7)
            seen.add(tuple(seq.tolist()))
            plain = ex.plain_log_probs(m, torch.cat([prompts[b], seq]), 9).sum()
            # both passes round every activation to bf16 (2^-8 of it); attention's sums differ in
            # their last fp32 bits, which flips few of those roundings: logits of size 10 may move by
            # a bf16 step of theirs, 2^-4, in some of the 12 tokens
            assert abs(float(plain) - float(score[b, k])) < 12 * 2.0 ** -4
        assert len(seen) == 3


def test_the_example_runs(ex, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["beam_decode.py", "--steps", "10", "--batch", "3"])
    ex.main()
    out = capsys.readouterr().out
    assert "student's loss on them" in out
