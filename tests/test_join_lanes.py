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


def test_a_wait_that_ran_out_leaves_nothing_under_way(common):
    """A thread whose wait ran out neither sends nor arrives any more: values sent ahead would count at a barrier for ones
    that are missing, and a second arrival in one phase is one too many.  The others' waits run out in their turn, and a
    CTA of which one ran out ends only some time after all of the cluster's have done so, when no store is under way."""
    write, meet, part = (body(common[common.index("struct Team"):], f"void {name}(") for name in ("write", "meet", "part"))
    assert re.search(r"if \(lane < ctas && !lost\)\s+asm volatile\(\"st\.async", write)
    assert re.search(r"if \(threadIdx\.x == 0 && !lost\) mbar_arrive_expect\(", meet)
    together, wait = part.index("this_cluster().sync()"), part.index("if (lost)")
    assert together < wait and re.search(r"while \(global_ns\(\) - start < kLandNs\);", part[wait:])
    assert 1_000_000 <= int(re.search(r"kLandNs = (\d+);", common).group(1)) <= 100_000_000
    assert common.count("st.async") == 1 and common.count("mbar_arrive_expect(") == 1
