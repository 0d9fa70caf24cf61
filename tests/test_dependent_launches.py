"""Kernels that are launched while the kernel before them ends read what it wrote by plain loads, which stay
behind the wait for it; the compiler may move read-only loads over that wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_attention_value_gb300", "csrc")


@pytest.mark.parametrize("name", ["append.cu", "attention.cu", "own.cu", "prefix.cu", "prefix.cuh"])
def test_no_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\s*\(|ld\.global\.nc|__restrict__", code)
