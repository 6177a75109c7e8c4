"""Rules that the sources of the 8-bit products and the router, and the code that they
compile to, have to keep whatever a build's register allocation looks like."""
import os
import re

from test_codegen import CSRC

SOURCES = {f: open(os.path.join(CSRC, f)).read() for f in sorted(os.listdir(CSRC)) if f.endswith((".hip", ".hpp"))}


def asm_blocks(text):
    """The inline assembly statements of a source, up to their semicolon."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            depth += 0 if quoted else (c == "(") - (c == ")")
            i += 1
        yield text[m.start():i]


def test_assembly_that_writes_m0_says_so():
    """The compiler keeps values of its own in M0 (indexed registers, its own direct loads); a
    block that changes it without naming it can take them away."""
    seen = 0
    for name, text in SOURCES.items():
        for block in asm_blocks(text):
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', block.split("::")[0]))
            if re.search(r"\b(?:s_mov_b32|s_add_u32|s_movk_i32)\s+m0\b", code):
                seen += 1
                assert block.rstrip().endswith('"m0")') or '"m0",' in block.rsplit(":", 1)[1], (name, block)
    assert seen >= 1


def test_matrix_core_calls_keep_their_operands():
    """Every call of a matrix-core builtin stands in a function that uses the result and both
    operands once more behind it, so that no allocation can place the result over an operand."""
    seen = 0
    for name, text in SOURCES.items():
        for m in re.finditer(r"__builtin_amdgcn_mfma_\w+\(", text):
            seen += 1
            rest = text[m.start():]
            body = rest[:rest.find("\n}\n")]
            assert re.search(r'keep_live\(r, a, b\);|asm\("" : "\+v"\(r\) : "v"\(a\), "v"\(b\)\);', body), (
                name, text.count("\n", 0, m.start()) + 1)
    assert seen >= 8
