"""Kernels that start before the one in front of them on the stream has ended (programmatic dependent launch) must read
what it writes through ordinary loads: the read-only path is for data that nothing writes while the kernel runs, and the
compiler may move such a load ahead of the wait."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_ternary_weight_b200", "csrc")


def text(path):
    """A source without its comments, with the project's headers that it includes."""
    with open(path) as f:
        s = f.read()
    s = re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)
    for name in re.findall(r'#include "([^"]+)"', s):
        if os.path.exists(os.path.join(CSRC, name)):
            s += text(os.path.join(CSRC, name))
    return s


WAITING = [os.path.basename(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if re.search(r"\bpdl_wait\(\);", text(p))]


def test_the_waiting_kernels_are_found():
    assert {"tern_norm.cu", "tern_kv4.cu", "tern_kv4_attn.cu", "tern_kv4_prompt.cu", "tern_gemm_i8.cu", "tern_gemv2.cu",
            "tern_gemv2w.cu", "tern_gemv3.cu"} <= set(WAITING)


@pytest.mark.parametrize("name", WAITING)
def test_no_read_only_loads(name):
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", text(os.path.join(CSRC, name)))
