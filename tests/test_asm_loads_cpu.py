"""Loads written in the kernels' inline assembly: no scalar register that they read comes straight from the compiler.

A vector memory instruction may read a scalar register only five instructions after a vector instruction (v_readlane,
v_readfirstlane) wrote it.  The compiler keeps that distance for its own loads, not for those inside assembly; a register
that a scalar instruction of the same assembly wrote is safe.
"""
import re

from tests.test_asm_clobbers_cpu import statements

LOAD = re.compile(r"\b(?:global|buffer|scratch|flat)_(?:load|store|atomic)\w*\s+(.*)")
SCALAR_WRITE = re.compile(r"\bs_(?:mov|add|sub|and|or|lshl|lshr|cselect)\w*\s+(%\d+)")


def operands(body):
    """(lines of code, constraint of each operand by number)."""
    parts = re.split(r'"\s*:', body, maxsplit=1)
    code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', parts[0] + '"')).replace("\\t", "")
    lists = parts[1].split(":") if len(parts) > 1 else []
    return code.split("\\n"), [c for part in lists[:2] for c in re.findall(r'"([^"]*)"\s*\(', part)]


def unsafe(body):
    """The loads' lines that read a scalar operand which no scalar instruction ahead of them wrote."""
    lines, kinds = operands(body)
    ours, bad = set(), []
    for line in lines:
        m = LOAD.search(line)
        if m:
            for n in re.findall(r"%(\d+)", m.group(1)):
                if "s" in kinds[int(n)] and f"%{n}" not in ours:
                    bad.append(line)
        m = SCALAR_WRITE.search(line)
        if m:
            ours.add(m.group(1))
    return bad


def test_bases_of_loads_are_written_beside_them():
    seen = 0
    for where, body in statements():
        seen += any(LOAD.search(line) for line in operands(body)[0])
        assert not unsafe(body), f"{where}: {unsafe(body)}"
    assert seen >= 2


def test_the_check_sees_a_base_from_outside():
    plain = '"s_mov_b64 exec, %2\\n\\tglobal_load_lds_dwordx4 %0, %1"::"v"(at), "s"(base), "s"(lanes) : "memory", "exec"'
    copied = '"s_mov_b64 %0, %2\\n\\tglobal_load_lds_dwordx4 %1, %0":"=&s"(from) : "v"(at), "s"(base) : "memory"'
    assert unsafe(plain) and not unsafe(copied)
