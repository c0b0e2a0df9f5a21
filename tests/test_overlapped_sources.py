"""Kernels launched to overlap the one before them (those that call pdl_wait) read nothing through
the read-only path.

Such a kernel may have started while its producer still writes, and a read-only load
(__ldg, ld.global.nc, or one that the compiler makes of a const __restrict__ pointer) promises data
that does not change from the kernel's start on.  Which loads the compiler makes of a
source cannot be seen in a result, so this reads the sources.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "parallelizable_recurrence_b200", "csrc")


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


OVERLAPPED = sorted(p for p in glob.glob(os.path.join(CSRC, "*.cuh")) if re.search(r"\bpdl_wait\(\);", _code(p)))


def test_the_sources_are_found():
    assert {"sru_cache.cuh", "sru_cache_attention.cuh", "sru_loss.cuh"} <= {os.path.basename(p) for p in OVERLAPPED}


@pytest.mark.parametrize("path", OVERLAPPED, ids=os.path.basename)
def test_no_read_only_loads(path):
    code = _code(path)
    for word in ("__ldg", "__restrict__", "ld.global.nc", "__ldlu"):
        assert word not in code, word


@pytest.mark.parametrize("path", OVERLAPPED, ids=os.path.basename)
def test_every_kernel_waits_before_its_first_load(path):
    """Each kernel calls pdl_wait once, and no pointer of its arguments is read before."""
    code = _code(path)
    bodies = re.split(r"__global__", code)[1:]
    assert bodies
    for body in bodies:
        body = body[body.index("{"):]
        assert body.count("pdl_wait();") == 1
        before = body[:body.index("pdl_wait();")]
        assert not re.search(r"\ba\.(targets|lse|dloss|lengths|table|slots|q|part|flags|offsets|n_free|add)\[", before)
        assert not re.search(r"\*a\.\w+", before)
