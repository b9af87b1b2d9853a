"""Kernels that fill their shared memory with bulk copies, by their source: a wait for a copy says whether it ran out, and
where it did the block waits for its copies once more, with a limit, before it goes on and leaves."""
import re

import pytest

from test_cluster_barrier_cpu import kernels

BULK = [k for k in kernels() if "bulk_copy_g2s(" in k[2]]


def test_they_are_found():
    assert "policy_rows_kernel" in {k[1] for k in BULK}


@pytest.mark.parametrize("file,name,body", BULK, ids=[k[1] for k in BULK])
def test_a_wait_that_ran_out_is_followed_by_another(file, name, body):
    assert "mbar_wait(" in body and not re.search(r"[;{})]\s*mbar_wait\(", body), "a wait's result is dropped"
    assert body.rindex("mbar_wait(") < body.index("mbar_drain(")
