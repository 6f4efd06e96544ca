"""The 8-bit cache's kernels and calls on a machine without a GPU: reads of what earlier kernels write."""

import glob
import os
import re

from conftest import ROOT


def test_nothing_is_read_as_unchanging():
    """A kernel with a programmatic launch lives while those before it still write lengths, tables, scales, lists, bounds and partial sums: none of
    these may be read as data that does not change while the kernel lives."""
    csrc = os.path.join(ROOT, "quantised_kv_cache_gb300", "csrc")
    files = glob.glob(os.path.join(csrc, "tq_q8*.cu*")) + [os.path.join(csrc, "tq_rotary.cu")]
    assert len(files) > 20
    for name in files:
        with open(name) as f:
            code = re.sub(r"//.*", "", f.read())
        assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", code), name
