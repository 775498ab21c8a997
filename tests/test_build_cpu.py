"""What the build needs and when it builds again (no compile of the CUDA
sources: their objects are there)."""
import os
import subprocess
import sys

import pytest

import __graft_entry__

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    __graft_entry__.build_library()


def run(code, *args):
    return subprocess.run([sys.executable, "-c", code] + [str(a) for a in args], cwd=ROOT, capture_output=True,
                          text=True, timeout=600)


WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None  # an import of torch fails
from speculative_decode_mla_tree_gb300 import build
build.LIB = sys.argv[1]
assert build.build() == sys.argv[1]
"""


def test_library_builds_without_torch(tmp_path):
    lib = tmp_path / "libmla_tree.so"
    r = run(WITHOUT_TORCH, lib)
    assert r.returncode == 0, r.stderr
    assert b"mla_tree_verify" in lib.read_bytes()


MODULE_FAILS = """
import sys
from speculative_decode_mla_tree_gb300 import build
build.LIB = sys.argv[1]
def fails():
    raise RuntimeError("no module")
build._compile_call = fails
try:
    build.build()
except RuntimeError as e:
    assert "no module" in str(e)
else:
    raise AssertionError("the failure is lost")
"""


def test_library_is_there_when_the_module_fails(tmp_path):
    lib = tmp_path / "libmla_tree.so"
    r = run(MODULE_FAILS, lib)
    assert r.returncode == 0, r.stderr
    assert lib.exists()
