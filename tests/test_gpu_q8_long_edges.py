"""Edges of the long-context calls of the 8-bit cache on the GPU: lists that take all of their blocks beside lists that choose, lists longer than
what their rows see."""

import numpy as np
import pytest
import torch

from quantised_kv_cache_gb300 import tq
from test_gpu_q8_attention import ints, make, np64
from test_gpu_q8_attention import queries as rows
from test_gpu_q8_blocks import BF, F32, HF, make_cache, queries, some_bounds, want_lists
from test_gpu_q8_sparse import check, poison_unlisted

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


@pytest.mark.parametrize("dtype", [BF, HF, F32])
# clusters of few rows, slices of them, warpgroups with units of their own, many rows in units of 256 and of 128
@pytest.mark.parametrize("B,Hq,H,n", [(1, 4, 1, 1), (200, 8, 1, 1), (200, 4, 1, 1), (4, 32, 4, 64), (40, 4, 4, 64)])
def test_lists_longer_than_what_is_seen(ctx, B, Hq, H, n, dtype):
    """Entries behind as many as there are seen blocks hold anything; a wrong one among these is passed over and reported."""
    r = np.random.default_rng(B)
    lens = r.integers(n, 129, B)
    cache, k, v = make(ctx, B, H, 640, lens.tolist(), seed=3, paged=B == 4)
    q = rows(5, B, Hq, n, dtype)
    named = np.full((B, H, 1, 9), -1, dtype=np.int32)
    named[..., :2] = [0, 1]
    lists = named.copy()
    lists[..., 2:] = [2 ** 31 - 1, 5, 5, -7, 3, 0, -2 ** 31]
    poison_unlisted(cache, named)
    lse = torch.empty(B, Hq, n, device=DEV)

    def call(x):
        out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
        tq.tq_q8_sparse_attention(ctx.handle, cache, torch.from_numpy(x).to(DEV), q, ints(lens), 640, span=n, lse=lse, out=out)
        return np64(out), tq.tq_get_device_error(ctx.handle)

    for x in (lists, named):
        got, error = call(x)
        assert error in ((0, tq.TQ_ERR_ARG) if x is lists else (0,))
        check(got, np64(q), k, v, named, n, lens, [n] * B, dtype=dtype, out_dtype=dtype, lse=np64(lse))
    lists[:, :, :, 0], lists[:, :, :, 1] = 1, 0  # not in order: the second is passed over
    got, error = call(lists)
    assert error == tq.TQ_ERR_ARG
    check(got, np64(q), k, v, np.where(named == 0, -1, named), n, lens, [n] * B, dtype=dtype, out_dtype=dtype, lse=np64(lse))
