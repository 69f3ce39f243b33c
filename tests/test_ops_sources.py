"""Rules that the operators' kernels keep and no run can show, read from their source.  No GPU."""

import os
import re

import pytest

from flow_matching_dit_b200.build import PKG

FILES = ("ops_attention.cuh", "ops_linear.cuh")


@pytest.mark.parametrize("name", FILES)
def test_a_warp_has_converged_before_a_lane_arrives_for_it(name):
    """In warps whose lanes each wait on a barrier for themselves, one lane's arrival speaks for the others: it lets the
    tensor core end the next phase, and a lane that still polls for the last one would then wait for ever.  So the
    statement in front of such an arrival is __syncwarp()."""
    src = open(os.path.join(PKG, "csrc", name)).read()
    lines = [re.sub(r"//.*", "", line).strip() for line in src.split("\n")]
    lines = [line for line in lines if line]
    found = 0
    for i, line in enumerate(lines):
        if re.search(r"if \(lane (== 0|< splits)\) mbar_arrive", line):
            found += 1
            assert lines[i - 1] == "__syncwarp();", "\n".join(lines[i - 3:i + 1])
    assert found >= 1


@pytest.mark.parametrize("name", FILES)
def test_kernels_that_wait_leave_after_their_copies(name):
    """A bounded wait that has run out lets a kernel's loops run to their end with copies into shared memory under way:
    each kernel whose waits are bounded gives them time to land before its CTAs leave."""
    src = open(os.path.join(PKG, "csrc", name)).read()
    kernels = re.findall(r"__global__ void.*?\n}\n", src, re.S)
    assert kernels
    for k in kernels:
        assert "op_wait" in k and k.count("op_leave(&s_abort)") == 1, k[:200]


def test_no_plain_static_is_written_after_it_was_made():
    """Calls run in several host threads at once: what the operators' host code keeps is const, atomic, behind a mutex or a
    thread's own."""
    for name in ("host.cuh", "ops.cu", "ops_common.cuh", "ops_linear.cuh", "ops_norm.cuh", "ops_attention.cuh"):
        for line in open(os.path.join(PKG, "csrc", name)).read().split("\n"):
            if re.match(r"\s+static (?!constexpr|const |__device__|_?_?inline)", line):
                assert re.search(r"std::(mutex|atomic|map|set)|int sms\[kMaxDevices\]", line), line   # (the last three under a mutex)
