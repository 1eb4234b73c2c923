"""The training and int8 entry points' host side under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU; host pass only, no GPU code is built), driven
by tests/sanitize/train_driver.cpp.  Built like test_sanitizers.py's library run."""
import concurrent.futures as cf
import glob
import os

import pytest

# (that file does not travel to machines that only run GPU tests)
_base = pytest.importorskip("test_sanitizers")
ENV, HERE, HIPCC, ROOT, SAN, _run = _base.ENV, _base.HERE, _base.HIPCC, _base.ROOT, _base.SAN, _base._run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_training_host_path_under_asan_ubsan(tmp_path):
    flags = ["--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-fPIC",
             "-Wno-unused-command-line-argument", "-w", "-I", os.path.join(ROOT, "include")]
    for f in SAN:
        flags += ["-Xarch_host", f]

    def cc(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, *flags, *(["-x", "hip"] if src.endswith(".cpp") else []), "-c", src, "-o", obj])
        return obj

    srcs = sorted(glob.glob(os.path.join(ROOT, "tile_level_gemm_02_amd", "csrc", "*.hip"))) + [os.path.join(HERE, "train_driver.cpp")]
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(cc, srcs))
    syms = {line.split()[-1] for o in objs for line in _run(["nm", "-u", o]).stdout.splitlines() if "__hip_fatbin_" in line}
    stub = tmp_path / "fatbin_stub.c"
    stub.write_text("".join(f'__attribute__((aligned(4096))) const char {s}[32] = "__CLANG_OFFLOAD_BUNDLE__";\n' for s in sorted(syms)))
    _run(["gcc", "-c", str(stub), "-o", str(tmp_path / "stub.o")])
    exe = str(tmp_path / "train_asan")
    _run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-Xarch_host", SAN[0], *objs, str(tmp_path / "stub.o"), "-o", exe])
    r = _run([exe], env=ENV, timeout=300)
    assert r.stdout.strip() == "ok", r.stdout[-3000:] + r.stderr[-3000:]
