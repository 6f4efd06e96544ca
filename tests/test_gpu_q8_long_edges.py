"""Edges of the long-context calls of the 8-bit cache on the GPU: lists that take all of their blocks beside lists that choose, lists longer than
what their rows see, queries that see nothing, captures side by side."""

import numpy as np
import pytest
import torch

from quantised_kv_cache_gb300 import tq
from test_gpu_q8_attention import ints, make, np64
from test_gpu_q8_attention import queries as rows
from test_gpu_q8_blocks import BF, F32, HF, make_cache, queries, some_bounds, want_lists
from test_gpu_q8_shared import caches
from test_gpu_q8_shared import check as check_shared
from test_gpu_q8_sparse import check, poison_unlisted, some_lists

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


# clusters of few rows, slices of them, warpgroups with units of their own (of one row and of more), many rows in units of 256 and of 128
SHAPES = [(4, 4, 1, 1), (200, 8, 1, 1), (200, 4, 1, 1), (90, 2, 2, 1), (6, 32, 4, 64), (40, 4, 4, 64)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("B,Hq,H,n", SHAPES)
def test_queries_of_sequences_without_tokens(ctx, B, Hq, H, n, dtype):
    """A query token of an empty sequence, or in front of a short one's first slot, is there: zeros, and a log-sum of -inf."""
    lens = np.random.default_rng(B).integers(0, 200, B)
    lens[::3], lens[1] = 0, 1
    cache, k, v = make(ctx, B, H, 256, lens.tolist(), seed=3)
    q = rows(5, B, Hq, n, dtype)
    lists = some_lists(B, H, 1, 4, np.full(B, 256), 3, 4)
    lse = torch.full((B, Hq, n), 7.0, device=DEV)
    got = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    tq.tq_q8_sparse_attention(ctx.handle, cache, torch.from_numpy(lists).to(DEV), q, ints(lens), 256, span=n, lse=lse, out=got)
    check(np64(got), np64(q), k, v, lists, n, lens, [n] * B, dtype=dtype, out_dtype=dtype, lse=np64(lse))
    assert not got[::3].any() and torch.isneginf(lse[::3]).all()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("B,Hq,H,n", SHAPES)
def test_prefixes_and_sequences_without_tokens(ctx, B, Hq, H, n, dtype):
    """The same behind a prefix: either part, or both, of some sequences empty."""
    r = np.random.default_rng(B)
    P = 150
    lens, prefix = r.integers(0, 200, B), r.integers(0, P + 1, B)
    lens[::3], prefix[::2] = 0, 0
    pre, own, pk, pv, k, v = caches(ctx, B, H, P, 256, lens.tolist(), 7)
    q = rows(5, B, Hq, n, dtype)
    lse = torch.full((B, Hq, n), 7.0, device=DEV)
    got = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    tq.tq_q8_shared_attention(ctx.handle, pre, ints(prefix), P, own, q, ints(lens), 256, lse=lse, out=got)
    check_shared(np64(got), np64(q), pk, pv, k, v, prefix, lens, [n] * B, dtype=dtype, out_dtype=dtype, lse=np64(lse))
    assert not got[::6].any() and torch.isneginf(lse[::6]).all()


def test_captures_side_by_side(ctx):
    """Two captures of each call with a workspace of its own, replayed at the same time on two streams, with other inputs every time: scores by
    the tensor cores (kept in the workspace), listed blocks and a prefix of many rows (partial records there)."""
    B, Hq, H, n, span, keep, cap, P = 2, 8, 2, 96, 32, 9, 64 * 150, 500
    lens = [cap, 5000]
    cache, e = make_cache(ctx, B, H, cap, seed=4)
    cache.tensors["v_stats"].view(F32).copy_(cache.tensors["k_stats"].view(F32))
    kv = [np64(x) for x in tq.tq_dequantize(ctx.handle, cache, 0, cap)]
    pre, own, pk, pv, k, v = caches(ctx, B, H, P, 256, [100, 200], 7)
    bounds, at, own_at, prefix = some_bounds(cache, 2), ints(lens), ints([100, 200]), ints([P, 300])
    size = max(tq.tq_q8_select_workspace(ctx.handle, B, Hq, H, n, span, cap), tq.tq_q8_sparse_attention_workspace(ctx.handle, B, Hq, H, n, span, keep),
               tq.tq_q8_shared_attention_workspace(ctx.handle, B, Hq, H, n, P, 256))
    assert tq.tq_q8_select_workspace(ctx.handle, B, Hq, H, n, span, cap) > 0

    class Side:
        def __init__(self, seed):
            self.seed, self.q, self.stream, self.graph = seed, rows(seed, B, Hq, n, BF), torch.cuda.Stream(), torch.cuda.CUDAGraph()
            self.blocks = torch.empty(B, H, n // span, keep, dtype=torch.int32, device=DEV)
            self.out, self.behind = torch.empty_like(self.q), torch.empty_like(self.q)
            self.workspace = ws = torch.empty(size, dtype=torch.uint8, device=DEV)
            with torch.cuda.graph(self.graph, stream=self.stream):
                for _ in range(3):
                    tq.tq_q8_select(ctx.handle, cache, bounds, self.q, at, cap, keep, sink=1, recent=1, span=span, workspace=ws, blocks=self.blocks)
                    tq.tq_q8_sparse_attention(ctx.handle, cache, self.blocks, self.q, at, cap, span=span, workspace=ws, out=self.out)
                    tq.tq_q8_shared_attention(ctx.handle, pre, prefix, P, own, self.q, own_at, 256, workspace=ws, out=self.behind)

    sides = [Side(5), Side(6)]
    for turn in range(3):
        for s in sides:
            s.q.copy_(rows(10 * turn + s.seed, B, Hq, n, BF))
            s.blocks.fill_(-7), s.out.fill_(7.0), s.behind.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(5):
            for s in sides:
                with torch.cuda.stream(s.stream):
                    s.graph.replay()
        torch.cuda.synchronize()
        for s in sides:
            lists = s.blocks.cpu().numpy()
            np.testing.assert_array_equal(lists, want_lists(cache, e, bounds, s.q, lens, None, span, keep, 1, 1))
            check(np64(s.out), np64(s.q), *kv, lists, span, lens, [n] * B, dtype=BF, out_dtype=BF)
            check_shared(np64(s.behind), np64(s.q), pk, pv, k, v, [P, 300], [100, 200], [n] * B, dtype=BF, out_dtype=BF)
