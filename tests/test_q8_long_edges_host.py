"""The 8-bit cache's kernels and long-context calls on a machine without a GPU: reads of what earlier kernels write, workspaces."""

import ctypes
import glob
import os
import re

import pytest
import torch

from conftest import ROOT
from quantised_kv_cache_gb300 import tq
from test_q8_blocks_host import pick
from test_q8_host import TAKEN, cache, ctx  # noqa: F401 (ctx: a fixture)


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


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would be enqueued")
@pytest.mark.parametrize("B,Hq,H,n,span,longest", [(1, 32, 8, 2048, 64, 16384), (1, 32, 8, 2048, 4, 16384), (3, 16, 2, 100, 33, 5000), (2, 8, 8, 40, 17, 64 * 33000),
                                                   (2, 8, 4, 1, 1, 64 * 40000), (5, 40, 2, 9, 1, 4096), (2, 4, 4, 3, 100, 64 * 40000)])
def test_a_choice_s_workspace_serves_smaller_calls_of_its_span(ctx, B, Hq, H, n, span, longest):  # noqa: F811
    def need(*a):
        size = ctypes.c_size_t()
        assert tq.lib().tq_q8_select_workspace(ctx, *a, ctypes.byref(size)) == 0
        return size.value

    most = need(B, Hq, H, n, span, longest)
    for b in sorted({1, B // 2 + 1, B}):
        for m in sorted({1, 2, 16 * H // Hq + 1, n // 3 + 1, n // 2 + 1, max(1, n - 1), n}):
            for length in (1, 64, longest // 3 + 1, longest - 1, longest):
                if m > n:
                    continue
                here = need(b, Hq, H, m, span, length)
                assert here <= most, (b, m, length)
                kw = dict(batch=b, heads_q=Hq, heads_kv=H, n_q=m, span=span, max_len=length, d_q=1 << 44, d_blocks=1 << 45)
                assert pick(ctx, cache(b, H, longest), ws_bytes=most, **kw) == TAKEN
                if here:  # what a call needs is what is asked for it
                    assert pick(ctx, cache(b, H, longest), ws_bytes=here - 1, **kw) == tq.TQ_ERR_WORKSPACE
    # another span has other lists: what it needs is checked, whatever the workspace was made for
    for other in (1, span // 2 + 1, 2 * span):
        here = need(B, Hq, H, n, other, longest)
        kw = dict(batch=B, heads_q=Hq, heads_kv=H, n_q=n, span=other, max_len=longest, d_q=1 << 44, d_blocks=1 << 45)
        assert pick(ctx, cache(B, H, longest), ws_bytes=most, **kw) == (TAKEN if here <= most else tq.TQ_ERR_WORKSPACE)
