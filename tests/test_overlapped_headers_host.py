"""Kernels that start while the launch before them still runs and stand in a
header: they take no read-only pointers either (see
test_overlapped_launches_host).  Read from the sources; no GPU needed."""

import glob
import os
import re

from test_overlapped_launches_host import CSRC, kernels


def test_kernels_in_headers_take_no_read_only_pointers():
    seen = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for name, params, body in kernels(text):
            if "griddep_wait" in body:
                seen.append(name)
                assert not re.search(r"const[^,]*__restrict__", params), f"{os.path.basename(path)}: {name}"
                # (and nothing that goes past coherence)
                assert "__ldg(" not in body and "ld.global.nc" not in body, name
    assert seen == ["residual_join_kernel"]
