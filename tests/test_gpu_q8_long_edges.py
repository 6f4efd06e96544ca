"""Edges of the long-context calls of the 8-bit cache on the GPU: lists that take all of their blocks beside lists that choose."""

import numpy as np
import pytest
import torch

from quantised_kv_cache_gb300 import tq
from test_gpu_q8_attention import ints
from test_gpu_q8_blocks import BF, make_cache, queries, some_bounds, want_lists

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantised_kv_cache_gb300 import build
    build.build()


@pytest.fixture()
def ctx():
    c = tq.Context(128, 8, "Q8", 1)
    yield c
    assert tq.tq_get_device_error(c.handle) == 0
    c.close()


@pytest.mark.parametrize("keep", [1, 5, 33, 100])
@pytest.mark.parametrize("B,blocks", [(2, 1024), (40, 300), (120, 150), (400, 150)])  # clusters of 8, 4, 2 and 1
def test_lists_of_all_blocks_in_clusters(ctx, B, blocks, keep):
    """`keep` no multiple of a warp: the lanes that write a list of all blocks leave the loop at different turns, with a cluster's barrier about."""
    cap = 64 * blocks
    cache, e = make_cache(ctx, B, 1, cap, seed=B, records=False)
    bounds = some_bounds(cache, keep)
    q = queries(B, 2, 1, BF, seed=keep)
    r = np.random.default_rng(keep)
    lens = r.integers(0, 64 * keep + 1, B)
    lens[::40] = cap - 64 * r.integers(0, 3, len(lens[::40]))
    out = torch.empty(B, 1, 1, keep, dtype=torch.int32, device=DEV)
    n = ints(lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(10):
            tq.tq_q8_select(ctx.handle, cache, bounds, q, n, cap, keep, blocks=out)
    want = want_lists(cache, e, bounds, q, lens.tolist(), None, 1, keep, 0, 1)
    for _ in range(20):
        out.fill_(-7)
        g.replay()
        np.testing.assert_array_equal(out.cpu().numpy(), want)
