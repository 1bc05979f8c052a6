"""Kernels that may start while the grid ahead of them still runs (no GPU: their source is read)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_flashattention_sdpa_gb300", "csrc")


@pytest.mark.parametrize("name", ["sdpa_pages.cu", "sdpa_verify.cu"])
def test_what_the_grid_ahead_writes_is_read_by_plain_loads(name):
    """Their inputs are any call's outputs, written while the kernel is already there: loads of data that does not change while a
    kernel lives (__ldg, .nc, pointers that are restrict) may be moved ahead of the wait."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//.*", "", f.read())
    assert "griddep_wait" in code
    assert not re.findall(r"__ldg\w*|\.nc\b|__restrict__|__ldca|__constant__", code)
