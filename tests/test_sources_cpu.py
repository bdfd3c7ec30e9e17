"""Rules of the kernel sources that no run can show."""
from __future__ import annotations

import glob
import os
import re

import pytest

from paged_kv_sliding_gb300.build import CSRC


def _code(path):
    text = open(path).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


OVERLAPPING = [os.path.basename(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
               if "grid_dependency_wait();" in _code(p)]


def test_the_overlapping_kernels_are_found():
    assert {"pkv_append.cu", "pkv_pages.cu", "pkv_decode_kernel.cuh", "pkv_prefill_kernel.cuh"} <= set(OVERLAPPING)


@pytest.mark.parametrize("name", OVERLAPPING)
def test_kernels_that_overlap_the_one_before_them_do_not_use_the_read_only_path(name):
    """That path (and a const __restrict__ pointer, which the compiler may take for it) asks
    that the data stays as it is for the kernel's whole life, which begins before the wait
    for the kernel that writes it; and such a load may be moved up across the wait."""
    code = _code(os.path.join(CSRC, name))
    assert not re.findall(r"__ldg\b|ld\.global(?:\.\w+)*\.nc|__restrict", code)
