"""What the linear-layer kernel does when a wait runs out, read in its source: on a device that works none does, and a
test must not make one hang.  A CTA may end only when nothing that reads or writes its memory is under way, and a part
of a sum that did not come must not be added up as if it had."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def roles():
    """The kernel's text by the warps' roles."""
    with open(os.path.join(ROOT, "bit_gradient_compression_gb300", "csrc", "linear.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    text = text[text.index("k_linear(const __grid_constant__"):text.index("k_linear_rows")]
    marks = ["if (warp == 0 && lane == 0)", "else if (warp == 1 && lane == 0", "else if (warp >= 4 && warp < 4 + S::kEpi)",
             "else if (warp >= 4 + S::kEpi)", "atomicAdd(&g_timeouts"]
    at = [text.index(m) for m in marks] + [len(text)]
    assert at == sorted(at)
    return dict(zip(("loads", "products", "epilogue", "loaders", "end"), (text[a:b] for a, b in zip(at, at[1:]))))


def after_loop(role):
    """What a role does behind its loop over tiles."""
    depth, i = 0, role.index("{", role.index("for (int64_t tile = worker"))
    while True:
        depth += {"{": 1, "}": -1}.get(role[i], 0)
        i += 1
        if depth == 0:
            return role[i:]


def test_every_wait_is_bounded(roles):
    for name, text in roles.items():
        for call in re.findall(r"(?:mbar|warp)_wait\(((?:[^()]|\([^()]*\))*)\)", text):
            assert call.endswith("p.wait_ns"), (name, call)
        assert "while (!mbar" not in text and "for (;;)" not in text


def test_loads_have_landed_and_been_read(roles):
    """The loading thread waits for the products on all of its stages, and for its copies where those do not come."""
    tail = after_loop(roles["loads"])
    wait, given_up = tail.index("mbar_wait(empty("), tail.index("if (gave_up)")
    assert wait < given_up < tail.index("mbar_wait(full(")
    assert "i < S::kStages" in tail[:wait]


def test_products_are_done(roles):
    """The thread that issues products waits for the last of them, whatever the epilogue does."""
    tail = after_loop(roles["products"])
    assert re.search(r"if \(!gave_up && ran\) gave_up = !mbar_wait\(acc_full\(", tail)
    given_up = tail[tail.index("if (gave_up)"):]
    assert given_up.index("mma_commit<PAIR>(drain)") < given_up.index("mbar_wait(drain")


def test_a_missing_part_is_nan(roles):
    """Before the CTAs of a cluster add up their parts, one that gave up makes its own NaN."""
    end = roles["end"]
    asked, nan = end.index("__syncthreads_or(gave_up)"), end.index("0x7FC00000u")
    assert asked < nan < end.index("cluster_sync()") < end.index("cluster_load8")
    assert re.search(r"for \(int i = threadIdx\.x; i < rows \* kTileM; i \+= S::kWarps \* 32\) st_shared4\(base", end)
