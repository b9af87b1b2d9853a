"""The losses without the decoding calls' CPython module: it builds, imports and runs without it."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def copy(tmp_path_factory):
    """The package with its built library, its sources no newer than that, and no module."""
    from conftest import build_lib
    build_lib()
    to = tmp_path_factory.mktemp("copy")
    pkg = os.path.join(ROOT, "output_projection_cross_gb300")
    shutil.copytree(pkg, to / "output_projection_cross_gb300",
                    ignore=lambda d, names: [n for n in names if n == "__pycache__" or n.startswith("_lossk_calls")
                                             or n.endswith(".o")])
    shutil.copytree(os.path.join(ROOT, "include"), to / "include")
    return to


def run(copy, script):
    r = subprocess.run([sys.executable, "-c", script], cwd=copy, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    return r


def test_the_module_is_named_for_its_python():
    from output_projection_cross_gb300 import build
    assert build.CALLS.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_the_losses_import_without_the_module(copy):
    run(copy, """
import output_projection_cross_gb300 as L, torch
assert L.__file__.startswith(%r), L.__file__
assert L.lossk_dims_check(4, 8, 16) == 580
assert L.lossk_decode_workspace_bytes(L.KIND_CACHE, 4, 16) > 0
try:
    L.lossk_beam_gather(torch.zeros(1, 2, 3), torch.zeros(1, 2, dtype=torch.int32), dst=torch.zeros(1, 2, 3),
                        ws=torch.zeros(256, dtype=torch.uint8))
    raise SystemExit("a decoding call without its module")
except ImportError as e:
    assert "build.py" in str(e)
""" % str(copy))


BUILD = """
import importlib.util, os, sysconfig
spec = importlib.util.spec_from_file_location("b", os.path.join("output_projection_cross_gb300", "build.py"))
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b._nvcc = lambda: (_ for _ in ()).throw(RuntimeError("the library is up to date"))
"""


def test_no_headers_of_python(copy):
    r = run(copy, BUILD + """
get = sysconfig.get_paths
sysconfig.get_paths = lambda *a: dict(get(*a), include="/nowhere")
b.build()
assert os.path.exists(b.LIB) and not os.path.exists(b.CALLS)
""")
    assert "Python.h" in r.stderr


def test_another_python_s_module_is_built_beside(copy):
    """A module that was built for another Python is neither loaded nor taken for this one's."""
    other = copy / "output_projection_cross_gb300" / "_build" / "_lossk_calls.cpython-39-other.so"
    other.write_bytes(b"not this Python's")
    run(copy, BUILD + "b.build(); assert os.path.exists(b.CALLS)")
    assert other.read_bytes() == b"not this Python's"
    run(copy, "import output_projection_cross_gb300.decode as d; assert d._calls.spans(None) == ()")
