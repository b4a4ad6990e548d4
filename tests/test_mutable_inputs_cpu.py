"""Kernels that start while the kernel before them still runs must not read its output by loads that take memory to be
constant for as long as the kernel lives."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "load_balanced_paged_02_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(x for x in os.listdir(CSRC) if x.endswith((".cu", ".cuh"))))
def test_plain_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    found = re.findall(r"__ldg\w*|ld\.global\.nc|const [\w ]+\*\s*__restrict__", code)
    assert not found, f"{name}: {found}"
