"""Kernels whose blocks reach into one another's shared memory, by their source: a cluster barrier says that every block of
the cluster has started before the first such access, and whoever arrives at it in two steps waits for it too."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "output_projection_cross_gb300", "csrc")


def kernels():
    """(file, name, body) of every kernel, comments left out."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path, encoding="utf-8") as fh:
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", fh.read(), flags=re.S)
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\([^{;]*\)\s*\{", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            yield os.path.basename(path), m.group(1), text[m.end():end]


REMOTE = [k for k in kernels() if "mapa_shared(" in k[2]]


def test_they_are_found():
    assert {k[1] for k in REMOTE} >= {"bwp_kernel", "fwd2_kernel", "policy_rows_kernel"}


@pytest.mark.parametrize("file,name,body", REMOTE, ids=[k[1] for k in REMOTE])
def test_a_barrier_comes_before_the_first_access(file, name, body):
    barrier = [m.start() for m in re.finditer(r"cluster_sync\(\)|cluster_wait_started\(\)", body)]
    assert barrier and barrier[0] < body.index("mapa_shared("), (file, name)


@pytest.mark.parametrize("file,name,body", REMOTE, ids=[k[1] for k in REMOTE])
def test_who_arrives_waits(file, name, body):
    if "cluster_arrive_started()" not in body:
        assert "cluster_wait_started()" not in body
        return
    at = body.index("cluster_arrive_started()")
    assert body.index("cluster_wait_started()") > at
    # every way out of the kernel up to the last wait has a wait just ahead of it
    last = body.rindex("cluster_wait_started()")
    for m in re.finditer(r"\breturn;", body[at:last]):
        assert re.search(r"cluster_wait_started\(\);\s*$", body[:at + m.start()]), (file, name)
