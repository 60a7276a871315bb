"""The kernels' inline assembly names every special register that it writes."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_routed_expert_amd", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\)\s*;", text, re.S):
            yield os.path.basename(path), m.group(1)


def test_written_registers_are_clobbers():
    seen = 0
    for where, body in statements():
        parts = re.split(r'"\s*:', body, maxsplit=1)
        code, rest = parts[0], parts[1] if len(parts) > 1 else ""
        for line in code.replace("\\t", "").split("\\n"):
            m = re.match(r'\s*"?\s*(\w+)\s+(m0|vcc|exec)\b', line)
            if m and m.group(1).startswith(("s_", "v_")):
                seen += 1
                assert f'"{m.group(2)}"' in rest, f"{where}: {line.strip()} writes {m.group(2)} and does not say so"
            if re.match(r'\s*"?\s*s_(add|sub|and|or|xor|lshl|lshr)', line):
                assert '"scc"' in rest, f"{where}: {line.strip()} writes scc and does not say so"
    assert seen
