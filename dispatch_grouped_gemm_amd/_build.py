"""Ahead-of-time build of libmoe_a8w4.so for gfx950 with hipcc, and of the binding's tensor
checks with the host compiler."""

from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe_a8w4.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.hip", "dispatch.hip", "quant.hip", "gemm_skinny.hip", "gemm_tiled.hip",
           "gemm_stream.hip", "combine.hip", "route.hip", "rows.hip", "adapter.hip",
           "ffn_forward.hip", "ffn_backward.hip", "norm.hip"]
CHECKS = os.path.join(HERE, "_checks.so")
CXX = os.environ.get("CXX", "g++")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # no packed fp32 instructions: ordinary float code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _checks_mark() -> bytes:
    """What _checks.so holds of the torch and the Python that it was built for."""
    import sys

    import torch
    return b"tensor checks for torch %s, %s\0" % (torch.__version__.encode(),
                                                  sys.implementation.cache_tag.encode())


def checks_current() -> bool:
    """Whether _checks.so is there and is this torch's and this Python's (it reads their
    structures, so it is not loaded to find out)."""
    try:
        with open(CHECKS, "rb") as f:
            return _checks_mark() in f.read()
    except OSError:
        return False


def _stale() -> bool:
    if not os.path.exists(LIB) or not checks_current():
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(CHECKS))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(HERE, "..", "include", "moe_a8w4.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def _build_checks() -> None:
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    tmp = CHECKS + ".tmp%d" % os.getpid()
    dirs = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           '-DCHECKS_MARK="%s"' % _checks_mark()[:-1].decode(),
           *["-isystem" + d for d in dirs], os.path.join(CSRC, "checks.cpp"), "-o", tmp,
           "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed for checks.cpp:\n%s%s" % (CXX, r.stdout, r.stderr))
    os.replace(tmp, CHECKS)


def build(force: bool = True, verbose: bool = False) -> str:
    """Compile every HIP source and link the shared library (in place)."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("hipcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        checks = ex.submit(_build_checks)
        objs = list(ex.map(compile_one, SOURCES))
        checks.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
