"""What the operators' sources must not hold (no GPU)."""
from __future__ import annotations

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gradient_ring_all_gb300", "csrc")


def test_no_read_only_loads():
    """Loads through the read-only path are defined only for memory that nobody
    writes while the kernel lives.  Under programmatic dependent launch a
    kernel is alive while the one before it still writes its inputs, and some
    kernels write the arrays that they read, so the library's kernels use
    ordinary loads alone."""
    found = []
    for folder, _, names in os.walk(CSRC):
        for name in names:
            text = open(os.path.join(folder, name)).read()
            found += ["%s: %s" % (name, m) for m in re.findall(r"__ldg\w*|ld\.global\.nc|__restrict__", text)]
    assert not found
