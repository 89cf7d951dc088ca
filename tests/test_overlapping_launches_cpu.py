"""Launches that may begin before the one before them has ended read nothing by the read-only path: it promises memory
that nobody writes while the kernel runs, and the compiler may move such loads past the wait."""
import glob
import os
import re

import pytest
from conftest import ROOT

CSRC = os.path.join(ROOT, "verify_gemm_gb300", "csrc")


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def overlapping():
    """The sources whose kernels wait for the launch before, and what they include of this folder but for the
    helpers that all kernels share."""
    files = {os.path.basename(p): code(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))}
    return sorted(n for n, s in files.items() if re.search(r"launch_before_has_ended\(\)|griddepcontrol\.wait", s))


def test_some_do():
    assert {"vg_attention.cuh", "vg_attention_wide.cuh", "vg_prefix.cu"} <= set(overlapping())


@pytest.mark.parametrize("name", overlapping())
def test_no_read_only_loads(name):
    s = code(os.path.join(CSRC, name))
    found = re.findall(r"__ldg\b|__restrict__|ld\.global\S*\.nc", s)
    assert not found, found
