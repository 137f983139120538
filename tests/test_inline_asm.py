"""Inline assembly of the kernels (no GPU): what a statement writes beyond its
outputs is declared, so that the compiler keeps nothing there."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "silent_corruption_detection_amd", "csrc")


def statements():
    """(file, instructions, clobbers) of every asm statement."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            parts = re.split(r":(?=(?:[^\"]*\"[^\"]*\")*[^\"]*$)", text[m.end():end - 1])
            code = "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", parts[0])).replace("\\n", "\n").replace("\\t", " ")
            clobbers = re.findall(r"\"([^\"]*)\"", parts[3]) if len(parts) > 3 else []
            out.append((os.path.basename(path), code, clobbers))
    return out


NAMED = r"(m0|vcc|exec|scc|[vsa]\d+|[vsa]\[\d+:\d+\])(_lo|_hi)?"


def test_written_registers_are_declared():
    """A register that an instruction names as its destination is a clobber."""
    for name, code, clobbers in statements():
        for line in code.splitlines():
            words = re.split(r"[\s,]+", line.strip())
            if len(words) > 1 and re.fullmatch(NAMED, words[1]):
                assert words[1] in clobbers, (name, code, clobbers)
            if words[0].startswith(("v_cmp", "s_cmp")):
                assert words[1].startswith("%") or {"vcc", "scc"} & set(clobbers), (name, code, clobbers)


def test_statements_are_found():
    found = statements()
    assert any("global_load_lds" in code for _, code, _ in found) and any("s_waitcnt" in code for _, code, _ in found)
