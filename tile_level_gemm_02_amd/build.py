"""Build libtg.so (the HIP kernels + C ABI) in-tree with hipcc for gfx950, and
the binding's native helper, _tgbind.so, with g++.

    python -m tile_level_gemm_02_amd.build          # or build() from Python

Each csrc/*.hip file is compiled to an object under _build/ (in parallel),
then linked into tile_level_gemm_02_amd/libtg.so.  The library needs neither
g++ nor torch's C++ headers; where the helper cannot be built, build() says so
in a warning and only the Python calls that need it are missing (tg_clip_grads,
tg_adamw, the int8 layers).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtg.so")
BIND = os.path.join(PKG, "_tgbind.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    # packed-FP32 VALU forms are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *CFLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build_bind() -> str:
    """Compile csrc/bind.cpp to _tgbind.so against torch's C++ headers (no GPU code); returns its path."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    inc = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"), *cpp_extension.include_paths()]
    libs = cpp_extension.library_paths()
    tmp = BIND + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{i}" for i in inc), os.path.join(CSRC, "bind.cpp"),
           *(f"-L{d}" for d in libs), "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    return BIND


def build(extra: list[str] | None = None, jobs: int | None = None) -> str:
    """Compile every HIP source and link libtg.so, and compile _tgbind.so beside it; returns libtg.so's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    extra = list(extra or [])
    jobs = jobs or min(len(srcs), max(1, (os.cpu_count() or 2)))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        bind = ex.submit(build_bind)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    try:
        bind.result()
    except Exception as e:  # no g++, no headers, or ones that bind.cpp does not fit
        if os.path.exists(BIND):
            os.remove(BIND)  # (of other sources or headers)
        warnings.warn(f"{BIND} was not built, tg_clip_grads, tg_adamw and the int8 layers cannot be called from Python: {e}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(sys.argv[1:]))
