"""Kernels that are launched chained (launch.cuh) may start before the kernel that writes what they read has ended. The read-only
path (ld.global.nc, __ldg, const __restrict__) is for memory that nothing writes during a kernel's life, so none of them takes it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "pack_virtual_rank_gb300", "csrc")
READ_ONLY = re.compile(r"\bld_stream_v4\b|\bMem<false>|\bload1<false>|\bld\.global\.nc\b|\b__ldg\b|\b__restrict__\b")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


CHAINED = sorted(n for n in os.listdir(CSRC) if n.endswith(".cu") and "launch_chained" in code(n))


def test_there_are_such_kernels():
    assert {"grads.cu", "fp8_quantize.cu", "grouped_router.cu", "router.cu", "head_rows.cu"} <= set(CHAINED)


@pytest.mark.parametrize("name", CHAINED)
def test_no_read_only_loads(name):
    own = set(re.findall(r'#include "(\w+\.cuh?)"', code(name))) - {"device.cuh"}     # device.cuh: the collectives' loads, too
    for part in [name] + sorted(own):
        found = READ_ONLY.findall(code(part))
        assert not found, (part, found)
