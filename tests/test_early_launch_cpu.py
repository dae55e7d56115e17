"""Kernels that may start while the kernel before them still runs read its
results: not through the read-only path, which wants data that nothing writes
while the kernel lives."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "second_order_post_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _early_sources():
    return [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "pdl_wait()" in _code(n)]


def test_there_are_some():
    assert {"dense.cu", "distill.cu"} <= set(_early_sources())


@pytest.mark.parametrize("name", _early_sources())
def test_no_read_only_loads(name):
    code = _code(name) + _code("act.cuh") + _code("common.cuh")
    assert not re.search(r"__ldg|ld\.global\.nc|\.nc\.|__restrict__", code)
