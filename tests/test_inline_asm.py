"""What the kernels' inline assembly writes is what it tells the compiler, on the CPU: scalar registers
that an instruction writes by name are in the statement's list of clobbered ones."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bf16_fp8_weight_amd", "csrc")


def _statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", text):
            depth, at = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[at], 0)
                at += 1
            yield os.path.basename(path), text[m.end():at - 1]


def test_registers_written_by_name_are_clobbered():
    seen = 0
    for name, statement in _statements():
        parts = re.split(r":(?=(?:[^\"]*\"[^\"]*\")*[^\"]*$)", statement)
        code, clobbers = parts[0], parts[-1] if len(parts) == 4 else ""
        for line in re.split(r"\\n\\t|\\n", code):
            words = line.strip().strip('"').split()
            if len(words) > 1 and words[0].startswith("s_") and words[1].rstrip(",") in ("m0", "vcc", "exec"):
                seen += 1
                assert f'"{words[1].rstrip(",")}"' in clobbers, f"{name}: {line}"
            if words and re.match(r"s_(add|sub|and|or|xor|cmp|lsh)", words[0]):
                assert '"scc"' in clobbers, f"{name}: {line}"
    assert seen >= 2
