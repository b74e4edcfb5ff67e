"""Kernels that start while the launch before them still runs
(griddepcontrol.wait) may not take read-only __restrict__ pointers: those
promise data that stays unchanged for the kernel's whole life, and allow reads
through the non-coherent path.  Read from the sources; no GPU needed."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_side_gb300",
                    "csrc")


def kernels(text):
    """(name, parameters, body) of every __global__ function."""
    for m in re.finditer(r"__global__\s+void[^;{]*?(\w+)\s*\(((?:[^(){};]|\([^()]*\))*)\)\s*\{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), m.group(2), text[m.end():at]


def test_kernels_that_start_early_take_no_read_only_pointers():
    seen = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for name, params, body in kernels(text):
            if "griddep_wait" in body:
                seen.append(name)
                assert not re.search(r"const[^,]*__restrict__", params), f"{os.path.basename(path)}: {name}"
    assert {"embed_sum_kernel", "embed_join_kernel"} <= set(seen)
