"""Properties of the token operators' sources that no run shows reliably."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "memory_bound_cnn_amd", "csrc")


def asm_statements():
    """(file, text, clobbers) of every extended asm statement of the token operators."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*tok*"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\);", src, flags=re.S):
            body = m.group(1)
            strings = r'"(?:[^"\\]|\\.)*"'
            text = re.match(rf"\s*((?:{strings}\s*)+)", body).group(1)
            rest = re.sub(rf"^\s*(?:{strings}\s*)+", "", body)
            # sections are ':' outside of parentheses and '::' of scope; clobbers are the third
            depth, parts = 0, [""]
            for c in rest.replace("::", ": :"):
                depth += (c in "([") - (c in ")]")
                if c == ":" and depth == 0:
                    parts.append("")
                else:
                    parts[-1] += c
            yield os.path.basename(path), text, re.findall(strings, parts[3]) if len(parts) > 3 else []


def test_inline_assembly_names_the_scalar_registers_it_writes():
    """A register that an asm statement writes and does not name may be one that
    the compiler keeps a value in."""
    seen = 0
    for name, text, clobbers in asm_statements():
        for reg in re.findall(r"\bs_\w+\s+(m0|vcc|exec|s\d+)\b", text):
            seen += 1
            assert f'"{reg}"' in clobbers, f"{name}: {text.strip()} writes {reg}, clobbers {clobbers}"
    assert seen > 0
