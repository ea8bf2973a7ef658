"""The plan's words, and the rows that are moved, are read with ordinary loads: a kernel that is resident before the one
that writes them has ended (programmatic launch) may not read them as constants of its whole run (__ldg, __restrict__)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "scaled_quantize_gemm_gb300", "csrc")
WORDS = r"(?:row_of|offsets|ntiles|tiles|blocks|plan|\bto\b)"


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", ["ffn_pair.cuh", "ffn_rows.cuh", "experts.cu", "experts_rows.cu"])
def test_no_constant_loads_of_plan_words(name):
    code = _code(name)
    assert not re.findall(rf"__ldg\((?:[^()]|\([^()]*\))*{WORDS}", code)
    assert not re.findall(rf"__restrict__\s+{WORDS}", code)
    loader = re.search(r"struct LoadPlan\s*\{.*?\};", code, re.S)
    assert loader is None or "__ldg" not in loader.group(0)


def test_no_constant_loads_of_rows():
    code = _code("experts_rows.cu")
    assert "__ldg" not in code
    assert not re.findall(r"const (?:V|T|float|int32_t)\* __restrict__", code)
