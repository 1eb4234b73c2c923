"""The LDS copies' descriptors in the built library (CPU: reads the listing).

The kernels issue their global-to-LDS copies from inline assembly.  A scalar
register written by a vector instruction (v_readfirstlane, v_readlane, a
compare) must not be read by a buffer instruction within five wait states; the
compiler sees to that for its own instructions but not inside inline assembly.
A first build of the weight gradient's kernel, whose descriptors move with the
K step, read stale descriptors that way."""
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WAIT_STATES = 5


def _scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"s(\d+)$", operand)
    return {int(m[1])} if m else {operand} if operand in ("m0", "vcc") else set()


def _hazards(lines):
    """(copies seen, [offending listing lines])"""
    history, copies, bad, name = [], 0, [], ""
    for line in lines:
        if line.endswith(">:\n"):
            history, name = [], line.strip()
            continue
        text = line.split("//")[0].strip()
        op, _, rest = text.partition(" ")
        if not op:
            continue
        operands = [o.strip() for o in re.split(r",\s*(?![^\[]*\])", rest)]
        if op.startswith("buffer_load") and rest.rstrip().endswith(" lds"):
            copies += 1
            need = _scalars(operands[1]) | _scalars(operands[2].split()[0]) | {"m0"}
            states = 0
            for before, args in reversed(history):
                if states >= WAIT_STATES:
                    break
                if before.startswith("v_") and _scalars(args[0]) & need:
                    bad.append(f"{name} {text} <- {before} {', '.join(args)}")
                    break
                states += int(args[0], 0) + 1 if before == "s_nop" else 1
        history.append((op, operands))
        del history[:-16]
    return copies, bad


def test_the_pattern_is_recognised():
    ok = "\tv_readfirstlane_b32 s8, v1\n\ts_nop 4\n\tbuffer_load_dwordx4 v2, s[8:11], s20 offen lds\n"
    late = "\tv_readfirstlane_b32 s8, v1\n\ts_nop 0\n\tbuffer_load_dwordx4 v2, s[8:11], s20 offen lds\n"
    other = "\tv_readfirstlane_b32 s12, v1\n\ts_nop 0\n\tbuffer_load_dwordx4 v2, s[8:11], s20 offen lds\n"
    assert _hazards(ok.splitlines(True)) == (1, [])
    assert _hazards(other.splitlines(True)) == (1, [])
    assert len(_hazards(late.splitlines(True))[1]) == 1
    assert len(_hazards(late.replace("s8,", "s20,").splitlines(True))[1]) == 1


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump not installed")
def test_no_copy_reads_a_scalar_too_soon(tmp_path):
    import tile_level_gemm_02_amd as tg

    lib = shutil.copy(tg.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    objects = [f for f in glob.glob(str(tmp_path / "*gfx950*")) if os.path.getsize(f)]
    assert objects
    total, bad = 0, []
    for f in objects:
        p = subprocess.Popen([OBJDUMP, "-d", "--no-show-raw-insn", f], stdout=subprocess.PIPE, text=True)
        copies, found = _hazards(p.stdout)
        assert p.wait() == 0
        total += copies
        bad += found
    assert total > 1000 and not bad, (total, bad[:5])
