"""Build liblcp.so (gfx950) in-tree from csrc/*.hip with hipcc, and _serve.so,
the marshalling of the serving calls, from csrc/bind.cpp with g++ (where that
fails, the build does, but liblcp.so is there for every other call).

    python learnable_channel_permutation_amd/build.py

Objects go to <repo>/_build/, the shared libraries next to this file. Every
invocation recompiles every source.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "liblcp.so")
BIND = os.path.join(PKG, "_serve.so")
ARCH = "gfx950"

# -packed-fp32-ops: keep fp32 arithmetic in plain (unpacked) VALU instructions.
HIPCC_FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


# Per-file extra flags. permute.hip does VALU work on every MFMA result; the
# VGPR form of MFMA keeps the accumulators out of AGPRs (no copy-out).
FILE_FLAGS = {"permute.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def _hipcc():
    for cand in ("/opt/rocm/bin/hipcc", "hipcc"):
        if os.path.isabs(cand) and os.path.exists(cand):
            return cand
    return "hipcc"


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src):
    obj = os.path.join(OBJ, os.path.basename(src)[:-4] + ".o")
    cmd = [_hipcc()] + HIPCC_FLAGS + FILE_FLAGS.get(os.path.basename(src), []) + ["-c", src, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, p.stderr))
    return obj


def _compile_bind():
    """csrc/bind.cpp against the headers of Python and torch, with torch's C++ ABI."""
    import torch as t
    torch = os.path.dirname(t.__file__)
    obj = os.path.join(OBJ, "host", "bind.o")        # apart from the library's objects
    os.makedirs(os.path.dirname(obj), exist_ok=True)
    abi = "-D_GLIBCXX_USE_CXX11_ABI=%d" % t.compiled_with_cxx11_abi()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", abi, "-isystem", os.path.join(torch, "include"), "-isystem",
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("g++ failed for bind.cpp:\n%s" % p.stderr)
    return obj, os.path.join(torch, "lib")


def _link_bind(obj, torch_lib):
    tmp = BIND + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-llcp", "-L", torch_lib, "-lc10", "-ltorch_cpu", "-ltorch",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("link of _serve.so failed:\n%s" % p.stderr)
    os.replace(tmp, BIND)


def build(verbose=False):
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    workers = min(len(srcs) + 1, int(os.environ.get("MAX_JOBS", "8")))
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        bind = ex.submit(_compile_bind)
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("link failed:\n%s" % p.stderr)
    os.replace(tmp, LIB)
    # after the library, which works without it, but not with an older one
    if os.path.exists(BIND):
        os.remove(BIND)
    _link_bind(*bind.result())
    if verbose:
        print("built", LIB, "and", BIND)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
