"""Build libssd.so (HIP, gfx950) in the package directory.

    python -m mamba_ssd_scan_05_amd.build

Each .hip source is compiled to an object by hipcc in parallel, then the
objects are linked into a shared library with a C ABI (include/ssd.h).  The
CPython module _pydesc (tensor descriptors for the Python binding) is built
beside it by g++ against torch's headers, where both are there.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libssd.so")
PYDESC = os.path.join(PKG, "_pydesc.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
SOURCES = ["ssd_api.hip", "ssd_kernels.hip", "ssd_prep.hip", "ssd_quad.hip", "ssd_rwalk.hip", "ssd_sscan.hip", "ssd_bwd.hip",
           "ssd_seq_api.hip", "ssd_glr.hip", "ssd_normrot.hip", "ssd_cache_api.hip", "ssd_append.hip", "ssd_attn.hip",
           "ssd_attn_rows.hip"]
# Per-source flags.  The row walk keeps its MFMA accumulators (the state
# tile) in ordinary VGPRs; otherwise the compiler places them in accumulator
# registers and copies them to VGPRs and back on every sub-block.  Likewise the
# scores of the attention's prompts (wide heads: N 256 775 -> 642 us).
EXTRA = {"ssd_rwalk.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
         "ssd_attn_rows.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}

COMMON = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
    # Keep the compiler from forming packed fp32 instructions.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Werror", "-Wno-unused-command-line-argument",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC] + COMMON + EXTRA.get(src, []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    return obj


def _compile_pydesc() -> bool:
    """Builds _pydesc where g++, Python's and torch's headers are there.  Where
    they are not, the binding packs its descriptors in Python; a module of an
    earlier build is taken out, since it may be of another torch."""
    cxx = os.environ.get("CXX", "g++")
    python_h = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    try:
        from torch.utils.cpp_extension import include_paths, library_paths
        torch_h = any(os.path.exists(os.path.join(d, "torch", "csrc", "autograd", "python_variable.h"))
                      for d in include_paths())
    except ImportError:
        torch_h = False
    missing = [n for n, there in ((cxx, shutil.which(cxx)), ("Python.h", os.path.exists(python_h)),
                                  ("torch's C++ headers", torch_h)) if not there]
    if missing:
        print("_pydesc is not built (no %s)" % ", ".join(missing), file=sys.stderr)
        if os.path.exists(PYDESC):
            os.remove(PYDESC)
        return False
    tmp = PYDESC + ".tmp%d" % os.getpid()
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           "-I" + os.path.join(ROOT, "include")]
    for d in include_paths() + [os.path.dirname(python_h)]:
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "ssd_pydesc.cpp"), "-o", tmp]
    for d in library_paths():  # torch's, loaded already when the module is imported
        cmd += ["-L" + d, "-Wl,-rpath," + d]
    cmd += ["-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed for ssd_pydesc.cpp:\n%s\n%s" % (cxx, " ".join(cmd), r.stderr))
    os.replace(tmp, PYDESC)
    return True


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        desc = ex.submit(_compile_pydesc)
        objs = list(ex.map(_compile, SOURCES))
        desc.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
