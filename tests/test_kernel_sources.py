"""What the kernels' sources have to say so that the compiler can hold them to it (no GPU, nothing is compiled)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_chunked_04_amd", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip")))


def code(path):
    """The file without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def statements(text):
    """Inline assembly: (instructions, operands and clobbers)."""
    for m in re.finditer(r"\basm\b\s*(?:volatile)?\s*\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        body = text[m.end():at - 1]
        instructions = re.match(r'\s*(?:"(?:[^"\\]|\\.)*"\s*)+', body).group(0)
        yield instructions, body[len(instructions):]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_assembly_leaves_m0_to_the_compiler(path):
    """The compiler keeps values of its own in M0 and cannot be told that a statement overwrites it: statements that need
    it there take it as an operand."""
    for instructions, operands in statements(code(path)):
        assert not re.search(r"\bm0\b", instructions, re.I), instructions
        if "load_lds" in instructions:
            assert '"{m0}"' in operands, instructions


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_helper_without_a_caller(path):
    everything = "\n".join(code(f) for f in FILES)
    for name in re.findall(r"__device__ __forceinline__ [^;{}()=]*?(\w+)\(", code(path)):
        assert len(re.findall(r"\b%s\b" % re.escape(name), everything)) > 1, name


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_wide_lds_accesses_are_declared_aligned(path):
    """An array in LDS that is read or written by 16 bytes says that it lies at a multiple of 16."""
    text = code(path)
    wide = set(re.findall(r"reinterpret_cast<(?:const )?(?:u32x4|f32x4)\s*\*>\(\s*&?\s*(\w+)\b", text))
    for declaration in re.findall(r"__shared__[^;]*;", text):
        for name in re.findall(r"(\w+)\s*\[", declaration):
            if name in wide:
                assert re.search(r"align(?:ed|__)\s*\(\s*\d+", declaration) or re.search(r"\b[uf]32x4\b", declaration), declaration
