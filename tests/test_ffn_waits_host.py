"""Waits of the dense feed-forward kernels that give up, read from the sources
(no GPU needed).  A lane that waits by itself finds out by itself that a wait
has given up, so lanes of a warp that each waited would part: some of them at
a warp's barrier or at a load from TMEM that the others never come to.  So
either one lane alone waits, or the warp votes; and a warp is in one piece
before each of the cluster's barriers, whose form is the aligned one."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_side_gb300",
                    "csrc")
IN_ONE_PIECE = r"(__syncwarp|__all_sync|__syncthreads)\([^;]*;"


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def blocks_around(text, at):
    """What stands before each of the braces that are open at a place, innermost first."""
    depth = 0
    for i in range(at - 1, -1, -1):
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth == 0:
                yield re.split(r"[;{}]", text[:i])[-1]
            else:
                depth -= 1


def test_lanes_do_not_part_at_a_wait():
    text = source("ffn.cu")
    waits = [m.start() for m in re.finditer(r"\bmbar_wait(_cluster)?\(", text)]
    assert len(waits) >= 7
    for at in waits:
        alone = any("lane == 0" in head for head in blocks_around(text, at))
        voted = text[:at].endswith("__all_sync(0xffffffffu, ")
        assert alone or voted, text[at - 200:at + 60]


def test_warps_come_to_the_clusters_barriers_in_one_piece():
    for name, most in (("ffn.cu", 5), ("ffn_rows.cu", 2)):
        text = source(name)
        calls = [m.start() for m in re.finditer(r"\bcluster_sync\(\)", text)]
        assert len(calls) == most
        for at in calls:
            whole = [m.end() for m in re.finditer(IN_ONE_PIECE, text[:at])][-1]
            # (nothing after it by which lanes part: no branch, no loop, no further wait)
            assert not re.search(r"\b(if|for|while|mbar_\w+)\b", text[whole:at]), text[whole:at]
