"""What the sources of the operators behind a router have to say to the compiler (no GPU needed)."""
import os
import re

import pytest

import top_selection_amd as ts
from test_expert_abi import _product

CSRC = os.path.join(os.path.dirname(ts.__file__), "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".h")))


def _asm(text):
    """(template, outputs and inputs, clobbers) of every inline assembly statement with operands."""
    for m in re.finditer(r"\basm(?:\s+volatile)?\s*\(((?:\"(?:[^\"\\]|\\.)*\"|[^\";])*)\)\s*;", text):
        body = m.group(1)
        template = "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", re.split(r"(?<!:):(?!:)|::", body)[0]))
        yield template, re.findall(r"\"((?:[^\"\\]|\\.)*)\"", body)


@pytest.mark.parametrize("name", SOURCES)
def test_registers_that_assembly_writes_are_declared(name):
    """m0 written by hand (where loads to LDS go) is the compiler's as well."""
    for template, strings in _asm(open(os.path.join(CSRC, name)).read()):
        if re.search(r"\bs_mov_b32 m0\b", template):
            assert "m0" in strings, f"{name}: {template}"


def test_the_reader_of_assembly_finds_the_loads():
    found = [t for t, _ in _asm(open(os.path.join(CSRC, "ds_product.hip")).read()) if "m0" in t]
    assert len(found) == 2


def test_exact_sums_are_asked_for_with_the_result_type():
    text = open(ts._binding.HEADER_PATH).read()
    assert int(re.search(r"#define DS_EXACT_SUMS (\d+)", text).group(1)) == ts.DS_EXACT_SUMS
    for otype in (ts.E4M3 | ts.DS_EXACT_SUMS, ts.DS_EXACT_SUMS << 1, -1):
        assert _product(otype=otype) == ts.DS_ERR_INVALID_ARG
    for otype in (ts.BF16, ts.FP32):  # the flag is no other type: its alignment is asked for
        assert _product(otype=otype | ts.DS_EXACT_SUMS, out=(8 << 40) + 1) == ts.DS_ERR_ALIGNMENT
    assert _product(otype=ts.FP32 | ts.DS_EXACT_SUMS, out=(8 << 40) + 2) == ts.DS_ERR_ALIGNMENT
    assert _product(otype=ts.BF16 | ts.DS_EXACT_SUMS, m=0, a=None, out=None) == 0
