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


OTHER_TORCH = """
import os, torch
from speculative_decode_mla_tree_gb300 import abi, build
here = build.call_path()
assert os.path.exists(here)
before = os.stat(here).st_mtime_ns
def differs(what):
    path = build.call_path()
    assert path != here and not os.path.exists(path), what
    abi._paged_call = None
    try:
        abi._load_paged_call()
    except abi.MlaTreeError as e:
        assert path in str(e)
    else:
        raise AssertionError(what + ": a module made for another was loaded")
for name in ("__version__", "version.git_version", "_C._GLIBCXX_USE_CXX11_ABI"):
    at, _, last = name.rpartition(".")
    holder = torch
    for part in at.split("."):
        holder = getattr(holder, part) if part else holder
    was = getattr(holder, last)
    setattr(holder, last, (not was) if isinstance(was, bool) else str(was) + ".other")
    differs(name)
    setattr(holder, last, was)
build.CALL_FLAGS.append("-DOTHER")
differs("flags")
build.CALL_FLAGS.pop()
suffix = build.sysconfig.get_config_var
build.sysconfig.get_config_var = lambda n: ".cpython-399-other.so" if n == "EXT_SUFFIX" else suffix(n)
differs("interpreter")
build.sysconfig.get_config_var = suffix
source = build.CALL_SRC
build.CALL_SRC = os.path.join(build.CSRC, "abi.cu")
differs("source")
build.CALL_SRC = source
assert build.call_path() == here and abi._load_paged_call()
assert os.stat(here).st_mtime_ns == before
"""


def test_module_of_another_torch_is_not_loaded():
    r = run(OTHER_TORCH)
    assert r.returncode == 0, r.stderr


BROKEN_LINK = """
import os, subprocess, sys
from speculative_decode_mla_tree_gb300 import build
build.LIBDIR = sys.argv[1]
def breaks_off(cmd, **kw):
    out = cmd[cmd.index("-o") + 1]
    open(out, "wb").write(b"half")
    assert out != build.call_path()
    return subprocess.CompletedProcess(cmd, 1, "", "killed")
build.subprocess = type("S", (), {"run": staticmethod(breaks_off)})
try:
    build._compile_call()
except RuntimeError as e:
    assert "killed" in str(e)
else:
    raise AssertionError("the failure is lost")
assert os.listdir(sys.argv[1]) == []
"""


def test_broken_link_leaves_no_module(tmp_path):
    r = run(BROKEN_LINK, tmp_path)
    assert r.returncode == 0, r.stderr
