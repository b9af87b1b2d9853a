"""The CPython module of the decoding calls: the same functions as through ctypes, argument by argument."""
import numpy as np
import pytest

import output_projection_cross_gb300 as L
from output_projection_cross_gb300 import decode

NAMES = ["lossk_beam_select", "lossk_beam_gather", "lossk_cache_fork", "lossk_cache_reserve", "lossk_cache_free",
         "lossk_cache_compact", "lossk_cache_copy", "lossk_cache_write", "lossk_paged_attn"]


def zeros(name):
    """Arguments that the call refuses on the host: zero sizes, no pointers."""
    c = {"c_void_p": None, "c_double": 0.0}
    return [c.get(t.__name__, 0) for t in getattr(L.lib, name).argtypes]


@pytest.mark.parametrize("name", NAMES)
def test_same_status_as_ctypes(name):
    args = zeros(name)
    assert getattr(decode._calls, name)(*args) == getattr(L.lib, name)(*args) != 580
    # every argument is the one of its place: a size after another turned to 1 changes both alike
    for i, a in enumerate(args):
        if a == 0 and not isinstance(a, float):
            args[i] = 1
            assert getattr(decode._calls, name)(*args) == getattr(L.lib, name)(*args) != 580


@pytest.mark.parametrize("name", NAMES)
def test_wrong_arguments(name):
    f, args = getattr(decode._calls, name), zeros(name)
    with pytest.raises(TypeError):
        f(*args[:-1])
    with pytest.raises(TypeError):
        f(*args, 0)
    with pytest.raises(TypeError):
        f("4", *args[1:])
    with pytest.raises(TypeError):
        f(1.5, *args[1:])
    with pytest.raises(OverflowError):
        f(1 << 64, *args[1:])
    assert f(np.int64(0), *args[1:]) == f(*args)


def test_a_code_out_of_range_is_no_other_code():
    args = zeros("lossk_beam_select")
    args[4] = (1 << 32) + 1                    # the type code is an int32
    with pytest.raises(OverflowError):
        decode._calls.lossk_beam_select(*args)


def test_spans_of_no_gpu_tensor():
    import torch
    spans = decode._calls.spans
    assert spans(torch.int32) == ()
    assert spans(torch.int32, None) == (0, 0)
    assert spans(torch.int32, None, torch.zeros(3, dtype=torch.int32)) is None     # not on a GPU
    assert spans(torch.int32, [1]) is None                                          # no tensor
    with pytest.raises(TypeError):
        spans()
