"""What orders the accesses of a warp's lanes to one another's places in shared memory, and what becomes of a wait that ran
out, in the join kernels: read in their source, as neither can be made to go wrong on a device by a test."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gradient_compression_gb300", "csrc")


@pytest.fixture(scope="module")
def common():
    with open(os.path.join(CSRC, "join_common.cuh")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, start):
    """The braces' content behind the first `start`."""
    i = text.index("{", text.index(start))
    depth, at = 0, i
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[at:i]


def test_lanes_meet_before_one_writes_into_anothers_place(common):
    """`load` writes the first bytes of the next lane's piece: not before that lane has read what was there for the last
    time, in the row before, and not where only some of the warp's lanes come."""
    load = body(common[common.index("struct Vec"):], "void load(")
    meet = load.index("if (ANY) __syncwarp();")
    assert meet < load.index("for (int e = 0") < load.index("copy_to_shared16") < load.index("place = piece(e, byte / 16)")
    # `settle` reads other lanes' pieces between two meetings
    settle = body(common[common.index("struct Vec"):], "void settle(")
    assert settle.index("if (ANY) __syncwarp();") < settle.index("ring16(piece(e, k))") < settle.index("to_ring16(piece(e, k)")
    assert settle.count("__syncwarp") == 2
