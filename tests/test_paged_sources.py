"""What the paged cache's sources must not hold, since no run would show it
reliably."""

import os
import re

from varlen_flashattention_backward_gb300 import build as fb


def code(name):
    with open(os.path.join(fb.CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_decode_reads_nothing_through_the_read_only_path():
    # The decode kernels may be on the GPU before the kernel that writes their lengths,
    # tables, rows and pages is done.  Non-coherent loads are defined for memory that
    # stays as it is for the whole life of the kernel that reads it.
    text = code("paged_decode.cuh")
    assert "griddepcontrol.wait" in text
    for load in ("__ldg", "ld.global.nc", ".nc.", "__restrict__"):
        assert load not in text, load
