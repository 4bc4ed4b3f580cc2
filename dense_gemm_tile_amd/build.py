"""Build libdense_gemm_tile_amd.so in-tree with hipcc for gfx950.

Usage: python dense_gemm_tile_amd/build.py [--incremental]
(or __graft_entry__.build(), which always compiles everything). It is
run as a script, not imported through the package, because importing the
package requires the library this script builds.
Objects go to _build/ at the repository root; the shared library and the
extension module that calls it (csrc/binding.cpp) land next to this file so the
Python binding finds them.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libdense_gemm_tile_amd.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BINDING_PATH = os.path.join(PKG_DIR, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (looked at $HIPCC, /opt/rocm/bin/hipcc, PATH)")


# Packed-FP32 VALU forms are switched off for every device pass.
COMMON_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")))


def _up_to_date(src: str, obj: str) -> bool:
    if not os.path.exists(obj):
        return False
    t = os.path.getmtime(obj)
    return all(os.path.getmtime(f) <= t for f in [src, *_headers()])


def _compile(src: str, extra, incremental: bool = False) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    if incremental and _up_to_date(src, obj):
        return obj
    cmd = [hipcc(), *COMMON_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _build_binding() -> None:
    """The extension module: host code only, linked to the library beside it. Without Python's
    headers it is left out (the package then calls the library through ctypes)."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        print(f"no Python.h in {include}: the extension module is left out", file=sys.stderr)
        if os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)  # of another build
        return
    tmp = BINDING_PATH + ".tmp"
    cmd = [hipcc(), "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
           "-no-hip-rt",
           "-I", os.path.join(ROOT, "include"), "-I", include,
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", PKG_DIR, f"-l:{LIB_NAME}",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"binding failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def build(verbose: bool = False, jobs: int | None = None, extra_flags=(),
          incremental: bool = False) -> str:
    """Compile every source (or, with incremental, those whose object is older
    than the source or any header) and link the library."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), max(1, min(16, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags), incremental), srcs))
    tmp = LIB_PATH + ".tmp"
    # -z defs: an undefined symbol (e.g. a kernel stub the compiler did not
    # emit) fails the link instead of the first dlopen.
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-z,defs", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _build_binding()
    if verbose:
        print(f"built {LIB_PATH} from {len(srcs)} sources", file=sys.stderr)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True, incremental="--incremental" in sys.argv[1:])
