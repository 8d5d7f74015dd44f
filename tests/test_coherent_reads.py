"""Kernels start before the one before them ends, and read what it wrote behind griddepcontrol.wait. That makes its writes visible to
coherent loads. The non-coherent path (__ldg) asks for data that stays constant while the kernel runs, which such data does not.
No run shows it, so the sources are read."""

import os
import re

import pytest

import rmsnorm_linear_projection_fold_b200 as fn

CSRC = os.path.join(os.path.dirname(fn.__file__), "csrc")


def _body(name, begin, end):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    return code[code.index(begin):code.index(end, code.index(begin))]


# kernels that are the first of a call, or follow one that lets them start before it has written what they read
@pytest.mark.parametrize("name,begin,end", [
    ("rope.cuh", "struct RopeVec", "struct RopeTableParams"),          # x and the table
    ("cross_entropy.cuh", " k_row_rstd(", "target_is_class"),
    ("cross_entropy.cuh", " k_ce_pack(", "struct CeGradParams"),        # lse, from the loss
    ("cross_entropy.cuh", " k_ce_dx(", "\n}\n\n}"),
    ("int8.cuh", " k_int8_rows(", "int8_swiglu"),
    ("decode_int8_cluster.cuh", " k_decode_int8_cluster(", "\n}\n\n}"),  # Q's scales, from the fold
])
def test_no_non_coherent_reads_of_what_the_kernel_before_wrote(name, begin, end):
    assert "__ldg(" not in _body(name, begin, end)


def test_the_fold_lets_no_pointer_be_read_that_way():
    """A const __restrict__ pointer without a cache operator tells the compiler the same as __ldg."""
    assert "__restrict__" not in _body("int8.cuh", " k_int8_scales(", "int8_take")
