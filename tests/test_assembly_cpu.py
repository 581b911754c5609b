"""No vector instruction is written as assembly in a source that runs matrix
instructions: the compiler keeps its own instructions clear of the registers that a
matrix instruction in flight still reads or writes, and adds no such waits for assembly.
Constants set before the first product are the exception."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "boolean_weight_amd", "csrc")
ASM = re.compile(r'\basm\s*(?:volatile\s*)?\(((?:\s*"(?:[^"\\]|\\.)*")+)')
VECTOR = re.compile(r"\bv_[a-z0-9_]+")


def read(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def sources(name, seen=None):
    """The file and the headers of this folder that it includes, with theirs."""
    seen = {} if seen is None else seen
    if name not in seen:
        seen[name] = text = read(name)
        for h in re.findall(r'#include "([^"/]+)"', text):
            sources(h, seen)
    return seen


@pytest.mark.parametrize("unit", sorted(f for f in os.listdir(CSRC) if f.endswith(".hip")))
def test_no_vector_assembly_beside_matrix_instructions(unit):
    files = sources(unit)
    if not any("__builtin_amdgcn_mfma" in t for t in files.values()):
        return
    found = [(name, op) for name, text in files.items() for a in ASM.findall(text)
             for op in VECTOR.findall(a) if op != "v_mov_b32"]
    assert not found


def test_it_finds_what_it_looks_for():
    a = ASM.findall('asm("v_bfi_b32 %0, %1" : "=v"(d)); asm volatile("s_nop 0\\n\\t" "v_add_u32 %0")')
    assert [VECTOR.findall(x) for x in a] == [["v_bfi_b32"], ["v_add_u32"]]
    assert ASM.findall(read("skinny.hip"))
