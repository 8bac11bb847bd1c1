"""What the cache kernels' sources must keep to, checked on their text and on their host-compiled arithmetic."""
import os
import re

import pytest

import pyramid_top_block_gb300 as pisa

CSRC = os.path.join(os.path.dirname(pisa.__file__), "csrc")


def code_of(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


EARLY = sorted(f for f in os.listdir(CSRC) if "griddepcontrol" in code_of(f) or "launch_early" in code_of(f))


def test_the_early_kernels_are_found():
    assert {"cache.cuh", "cache_append.cu", "cache_attend.cuh"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_kernels_that_start_early_load_coherently(name):
    """A kernel that starts while the one before it still writes may not use the read-only path: such a load
    promises that nothing writes the memory while the kernel lives, and may move ahead of the wait."""
    found = re.findall(r"__ldg\b|\bld\.global(?:\.\w+)*\.nc\b|__restrict__|__ldlu\b", code_of(name))
    assert not found, found
