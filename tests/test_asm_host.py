"""Host-side check of the sources' inline assembly: what a statement writes beside its operands it says."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nested_bit_weight_amd", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"\basm\s+(?:volatile\s*)?\(", text):
            depth, at = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[at], 0)
                at += 1
            yield f"{os.path.basename(path)}:{text.count(chr(10), 0, m.start()) + 1}", text[m.end():at - 1]


def code_and_clobbers(body):
    """The instructions of a statement, and what stands after its third colon."""
    strings = r'(?:"(?:[^"\\]|\\.)*"\s*)+'
    code = re.match(r"\s*" + strings, body).group(0)
    rest = re.sub(r'"(?:[^"\\]|\\.)*"', lambda s: s.group(0).replace(":", ";"), body[len(code):])
    parts = rest.replace("::", ": :").split(":")
    return code, parts[3] if len(parts) > 3 else ""


def test_registers_that_inline_assembly_writes_are_named():
    found = 0
    for where, body in statements():
        code, clobbers = code_and_clobbers(body)
        found += 1
        for register in ("m0", "vcc", "scc", "exec"):
            if re.search(r"\bs_\w+\s+" + register + r"\b", code):
                assert f'"{register}"' in clobbers, (where, register)
    assert found > 5
