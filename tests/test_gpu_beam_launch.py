"""Selections whose launches a process makes first: sizes on either side of the shared memory a kernel has
without asking, and what a call finds on a workspace that another call left.

Each script runs in a process of its own, for a larger selection before it would raise the limits.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

START = """
import torch
import output_projection_cross_gb300 as L
g = torch.Generator(device="cuda").manual_seed(1)

def inputs(B, K, V):
    return (torch.randn(B * K, V, device="cuda", generator=g).bfloat16(),
            -torch.rand(B, K, device="cuda", generator=g))
"""


def run(script):
    from conftest import build_lib
    build_lib()
    r = subprocess.run([sys.executable, "-c", START + script], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_call_after_one_that_was_refused():
    """512 rows are more than the rows kernel has blocks: which rows it takes hangs on its counter."""
    run("""
B, K, V = 16, 32, 32000
ws = L.decode_workspace(L.KIND_BEAM_SELECT, B, K, V, 64)
x, s = inputs(B, K, V)
try:
    L.lossk_beam_select(x, s, 64, ws=ws)
except L.LosskError:
    pass
for n in (8, 3):
    x, s = inputs(B, K, V)
    got = L.lossk_beam_select(x, s, n, ws=ws)
    want = L.lossk_beam_select(x, s, n)
    assert all(torch.equal(got[k], want[k]) for k in got)
    rank = (s.double()[:, :, None] + torch.log_softmax(x.double(), -1).view(B, K, V)).view(B, -1)
    assert torch.equal(rank.topk(n).indices, got["parent"].long() * V + got["token"])
assert L.lossk_device_status(ws) == 580
""")


@pytest.mark.parametrize("B,K,V,n", [
    # the merge takes 24 bytes a candidate, or 128 an entry of a beam's split lists: on both sides of 48 KB
    # less its own arrays (45 to 46 KB), and of 48 KB
    (64, 32, 151936, 64), (16, 32, 32000, 64), (1, 12, 128256, 24), (1, 9, 151936, 18), (2000, 30, 513, 64),
    (2000, 30, 513, 63), (2000, 31, 513, 62), (700, 15, 600, 128), (700, 17, 600, 128)])
def test_sizes_about_the_limit_as_a_process_first_call(B, K, V, n):
    run(f"B, K, V, n = {B}, {K}, {V}, {n}" + """
x, s = inputs(B, K, V)
ws = L.decode_workspace(L.KIND_BEAM_SELECT, B, K, V, n)
got = L.lossk_beam_select(x, s, n, ws=ws)
assert L.lossk_device_status(ws) == 580
for b in (0, B // 2, B - 1):
    rows = x[b * K:(b + 1) * K].double()
    rank = (s[b].double()[:, None] + torch.log_softmax(rows, -1)).view(-1)
    best = rank.topk(n + 1).values
    at = got["parent"][b].long() * V + got["token"][b]
    # (bf16 logits tie: candidates of equal rank may stand in another order here; a score's rounding is
    # 2^-24 of 20 and its log-sum-exp's error 3e-6)
    assert torch.allclose(rank[at], best[:n], rtol=0, atol=1e-5) and len(set(at.tolist())) == n
    assert torch.allclose(got["score"][b].double(), best[:n], rtol=0, atol=1e-5)
""")


def test_a_process_first_calls_recorded_into_a_graph():
    """Whatever a kernel's first launch needs is done while the stream records."""
    run("""
x, s = inputs(2, 4, 20001)
y, s2 = inputs(3, 5, 77)
ws, out = L.decode_workspace(L.KIND_BEAM_SELECT, 2, 4, 20001, 8), L.beam_buffers(2, 8)
ws2, out2 = L.decode_workspace(L.KIND_BEAM_SELECT, 3, 5, 77, 8), L.beam_buffers(3, 8)
cases = []
for dt in (torch.bfloat16, torch.float16, torch.float32):
    k, v = (torch.randn(40, 16, 2, 64, device="cuda", generator=g).to(dt) for _ in range(2))
    q = torch.randn(4, 8, 64, device="cuda", generator=g).to(dt)
    t = torch.randperm(40, device="cuda", generator=g).int().view(4, 10)
    cases.append((q, k, v, t, torch.tensor([160, 1, 77, 33], dtype=torch.int32, device="cuda")))
wa = [L.decode_workspace(L.KIND_PAGED_ATTN, 4, 8, 2, 64) for _ in cases]
o = [torch.zeros_like(c[0]) for c in cases]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    L.lossk_beam_select(x, s, 8, out=out, ws=ws)
    L.lossk_beam_select(y, s2, 8, out=out2, ws=ws2)
    for c, w, a in zip(cases, wa, o):
        L.lossk_paged_attn(*c, share=2, out=a, ws=w)
graph.replay()
torch.cuda.synchronize()
for a, b in ((out, L.lossk_beam_select(x, s, 8)), (out2, L.lossk_beam_select(y, s2, 8))):
    assert all(torch.equal(a[n], b[n]) for n in a)
for c, a in zip(cases, o):
    assert torch.equal(a, L.lossk_paged_attn(*c, share=2))
""")
