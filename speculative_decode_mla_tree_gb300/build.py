"""Compile the CUDA library in tree: every csrc/*.cu for sm_103a, linked
into lib/libmla_tree.so (static CUDA runtime; needs nvcc and nothing else), and,
where torch is installed, csrc/paged_call.cpp, the paged calls' way in from
Python tensors, into a lib/_paged_call.*.so (see call_path). Translation units
compile in parallel; a unit is rebuilt only when a source or header is newer
than its object file."""
from __future__ import annotations

import glob
import hashlib
import os
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
OBJDIR = os.path.join(LIBDIR, "obj")
LIB = os.path.join(LIBDIR, "libmla_tree.so")
CALL_SRC = os.path.join(CSRC, "paged_call.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]


def nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _compile(src, ptxas_verbose=False):
    obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
    newest = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest and not ptxas_verbose:
        return obj, ""
    cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    return obj, r.stderr


CALL_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared"]
CALL_LIBS = ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _abi_flag():
    import torch
    return "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)


def call_path():
    """Where the extension module for this interpreter and this torch is, or will
    be built. It reads tensors' fields where torch's headers put them, so its
    name tells the interpreter's ABI, torch's version, the flags and the sources
    apart: one that was made for anything else is never loaded."""
    import torch
    h = hashlib.sha256()
    for part in [torch.__version__, str(torch.version.git_version), _abi_flag()] + CALL_FLAGS + CALL_LIBS:
        h.update(part.encode() + b"\0")
    for path in (CALL_SRC, os.path.join(ROOT, "include", "mla_tree.h")):
        with open(path, "rb") as f:
            h.update(f.read() + b"\0")
    return os.path.join(LIBDIR, "_paged_call.%s%s" % (h.hexdigest()[:16], sysconfig.get_config_var("EXT_SUFFIX")))


def _compile_call():
    """The extension module, against this interpreter's headers and torch's;
    None without torch, whose tensors are all that it is for."""
    try:
        import torch
    except ImportError:
        return None
    path = call_path()
    if os.path.exists(path):
        return path
    part = "%s.%d.part" % (path, os.getpid())  # a link that breaks off leaves nothing that looks whole
    t = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda", "include")
    cmd = ["g++"] + CALL_FLAGS + [_abi_flag(), "-I" + sysconfig.get_paths()["include"],
                                  "-I" + os.path.join(t, "include"),
                                  "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"), "-I" + cuda,
                                  CALL_SRC, "-o", part, "-L" + os.path.join(t, "lib")] + CALL_LIBS
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(part):
            os.remove(part)
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (CALL_SRC, " ".join(cmd), r.stderr))
    os.replace(part, path)
    return path


def build(verbose=False, ptxas_verbose=False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        call = ex.submit(_compile_call)
        results = list(ex.map(lambda s: _compile(s, ptxas_verbose), srcs))
    objs = [o for o, _ in results]
    if verbose or ptxas_verbose:
        for (o, log) in results:
            if log:
                print(log)
    if (not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        cmd = [nvcc()] + ARCH + ["-shared", "-o", LIB] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    call.result()  # what failed there is raised once the library is in place
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, ptxas_verbose="-v" in sys.argv))
