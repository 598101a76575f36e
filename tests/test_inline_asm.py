"""Inline assembly tells the compiler what it changes: the register m0 where
it is written, and memory where the instruction reads or writes it."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOUCHES_MEMORY = re.compile(
    r"\b(buffer|global|flat|ds|scratch)_|\blds\b|s_barrier|s_waitcnt")


def blocks():
    for path in sorted(glob.glob(os.path.join(
            ROOT, "fp8_mx_activation_amd", "csrc", "*"))):
        src = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", src):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(src[i], 0)
                i += 1
            body = src[m.end():i - 1]
            parts = re.split(r":(?=(?:[^\"]*\"[^\"]*\")*[^\"]*$)", body)
            yield (os.path.basename(path), parts[0],
                   parts[3] if len(parts) > 3 else "")


def test_asm_names_what_it_changes():
    seen = 0
    for name, code, clobbers in blocks():
        seen += 1
        if re.search(r"\bm0\b", code):
            assert '"m0"' in clobbers, (name, code)
        if TOUCHES_MEMORY.search(code):
            assert '"memory"' in clobbers, (name, code)
    assert seen > 0
