"""Rules that the sources of the 8-bit products and the router, and the code that they
compile to, have to keep whatever a build's register allocation looks like."""
import os
import re

import pytest

from test_codegen import CSRC, HIPCC, _all_asm

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


def kernels(source):
    """(name, lines of assembly) of a source's kernels."""
    srcs, asms = _all_asm()
    text = dict(zip([os.path.basename(s) for s in srcs], asms))[source]
    for m in re.finditer(r"^(_Z\w+):.*?^\s*s_endpgm.*?^\.Lfunc_end\d+:", text, re.M | re.S):
        lines = [line.split(";")[0].strip() for line in m.group(0).splitlines()]
        yield m.group(1), [line for line in lines if line and not line.startswith(".")]


needs_hipcc = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@needs_hipcc
def test_joined_shares_are_released_and_acquired():
    """The workgroups' shares of the balance loss are written before the ticket that hands them over
    and read behind it by the memory model's own means: a release (the cache written back) in front of
    the ticket, an acquire (the cache invalidated) behind it."""
    code = [lines for name, lines in kernels("route.hip") if "route_join_kernel" in name]
    assert len(code) == 1
    at = [i for i, line in enumerate(code[0]) if line.startswith("global_atomic_add")]
    assert len(at) == 1
    before, behind = code[0][:at[0]], code[0][at[0]:]
    assert any(line.startswith("buffer_wbl2") and "sc1" in line for line in before)
    assert any(line.startswith("buffer_inv") and "sc1" in line for line in behind)


@needs_hipcc
@pytest.mark.parametrize("source", ["route.hip", "w8a8.hip"])
def test_shared_memory_is_accessed_as_such(source):
    """No access through generic addresses: one waits for every outstanding load of its wave and
    says nothing about the order of shared memory."""
    for name, lines in kernels(source):
        bad = [line for line in lines if line.startswith("flat_")]
        assert not bad, (name, len(bad), bad[:3])


@needs_hipcc
@pytest.mark.parametrize("source", ["route.hip", "w8a8.hip"])
def test_nothing_is_spilled(source):
    srcs, asms = _all_asm()
    text = dict(zip([os.path.basename(s) for s in srcs], asms))[source]
    sizes = re.findall(r"\.amdhsa_private_segment_fixed_size (\d+)", text)
    assert len(sizes) > 10 and set(sizes) == {"0"}
