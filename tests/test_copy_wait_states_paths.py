"""The LDS copies' descriptors along every path of the built library's code
(CPU: reads the listing).

test_copy_wait_states.py looks at the instructions listed ahead of a copy.  A
register can also be written at the end of a loop's body and read by a copy at
its head, or on the far side of any other branch: here the five wait states
are followed backwards along the control flow, through every branch that leads
to an instruction as well as through the one listed before it."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from test_copy_wait_states import OBJDUMP, WAIT_STATES, _scalars

_LINE = re.compile(r"\s*(\S+)\s*(.*?)\s*//\s*([0-9A-Fa-f]+):.*?(?:<[^>+]*(?:\+0x([0-9a-f]+))?>)?\s*$")
_HEAD = re.compile(r"([0-9a-f]+) <(.*)>:")
_STOPS = ("s_branch", "s_endpgm", "s_setpc_b64")


def _functions(lines):
    """(name, [(address, op, operands, branch target or None)]) of a listing."""
    name, base, code = None, 0, []
    for line in lines:
        m = _HEAD.match(line)
        if m:
            if code:
                yield name, code
            name, base, code = m[2], int(m[1], 16), []
            continue
        m = _LINE.match(line) if name else None
        if m:
            operands = [o.strip() for o in re.split(r",\s*(?![^\[]*\])", m[2])]
            target = None
            if m[1].startswith(("s_branch", "s_cbranch")):
                target = base + (int(m[4], 16) if m[4] else 0)
            code.append((int(m[3], 16), m[1], operands, target))
    if code:
        yield name, code


def _written(op, operands):
    """Scalar registers that a vector instruction writes."""
    if not op.startswith("v_"):
        return set()
    out = _scalars(operands[0])
    if len(operands) > 1 and ("_co_" in op or "div_scale" in op or op.startswith(("v_mad_u64", "v_mad_i64"))):
        out |= _scalars(operands[1])
    return out


def _path_hazards(code):
    """(copies, [offending instructions]) of one function."""
    at = {c[0]: i for i, c in enumerate(code)}
    before = [[i - 1] if i and not code[i - 1][1].startswith(_STOPS) else [] for i in range(len(code))]
    for i, (_, _, _, target) in enumerate(code):
        if target is not None:
            before[at[target]].append(i)
    copies, bad = 0, []
    for i, (_, op, operands, _) in enumerate(code):
        if not (op.startswith("buffer_load") and operands[-1].endswith(" lds")):
            continue
        copies += 1
        need = _scalars(operands[1]) | _scalars(operands[2].split()[0]) | {"m0"}
        work, seen = [(p, 0) for p in before[i]], {}
        while work:
            p, states = work.pop()
            if states >= WAIT_STATES or seen.get(p, WAIT_STATES) <= states:
                continue
            seen[p] = states
            _, o, args, _ = code[p]
            if _written(o, args) & need:
                bad.append(f"{op} {', '.join(operands)} <- {o} {', '.join(args)}")
                break
            states += int(args[0], 0) + 1 if o == "s_nop" else 1
            work += [(q, states) for q in before[p]]
    return copies, bad


def _found(*rows):
    """_path_hazards of a function of 4-byte instructions: (text, index of the branch's target)."""
    lines = ["0000000000001000 <f>:\n"]
    for i, (text, to) in enumerate(rows):
        where = "" if to is None else " <f>" if to == 0 else f" <f+{4 * to:#x}>"
        lines.append(f"\t{text:60s}// {0x1000 + 4 * i:012X}: 00000000{where}\n")
    (_, code), = _functions(lines)
    assert len(code) == len(rows)
    return _path_hazards(code)


COPY = ("buffer_load_dwordx4 v2, s[8:11], s20 offen lds", None)
WRITE = ("v_readfirstlane_b32 s8, v1", None)
WAIT, END = ("s_nop 4", None), ("s_endpgm", None)


def test_paths_are_followed():
    assert _found(WRITE, WAIT, COPY, END) == (1, [])
    assert len(_found(WRITE, COPY, END)[1]) == 1
    # written at the end of a loop's body, read at its head
    back = ("s_cbranch_scc1 65531", 0)
    assert len(_found(COPY, ("s_nop 7", None), WRITE, back, END)[1]) == 1
    assert _found(COPY, ("s_nop 7", None), WRITE, WAIT, back, END) == (1, [])
    # a jump over the wait
    assert len(_found(WRITE, ("s_branch 1", 3), ("s_nop 7", None), COPY, END)[1]) == 1
    # what is listed before the copy does not lead to it
    assert _found(("s_cbranch_scc0 2", 3), WRITE, END, COPY, END) == (1, [])
    # a carry written to the descriptor
    assert len(_found(("v_add_co_u32_e64 v1, s[8:9], v2, v3", None), COPY, END)[1]) == 1


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump not installed")
def test_no_copy_reads_a_scalar_too_soon_on_any_path(tmp_path):
    import tile_level_gemm_02_amd as tg

    lib = shutil.copy(tg.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    objects = [f for f in glob.glob(str(tmp_path / "*gfx950*")) if os.path.getsize(f)]
    assert objects
    copies, branches, bad = 0, 0, []
    for f in objects:
        p = subprocess.Popen([OBJDUMP, "-d", f], stdout=subprocess.PIPE, text=True)
        for name, code in _functions(p.stdout):
            n, found = _path_hazards(code)
            copies += n
            branches += sum(c[3] is not None for c in code)
            bad += [f"{name}: {b}" for b in found]
        assert p.wait() == 0
    assert copies > 1000 and branches > 1000 and not bad, (copies, branches, len(bad), bad[:5])
