"""Attention of a batch behind a shared prefix on the GPU, against fp64 attention over the prefix's and the sequences' own values one after
the other (oracle/q8_blocks.py), within the bound of tests/q8_rows.py."""

import numpy as np
import pytest
import torch

from q8_rows import BF, F32, HF, assert_rows
from quantised_kv_cache_gb300 import tq
from test_gpu_q8_attention import gen, ints, make, np64, queries

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


def check(got, q, pk, pv, k, v, prefix, lens, new, *, dtype, out_dtype, begin=None, end=None, slopes=None, lse=None, **kw):
    B, Hq, n, _ = q.shape
    H = k.shape[1]
    G = Hq // H
    worst = 0.0
    for b in range(B):
        P, L, m = int(prefix[b]), int(lens[b]), int(new[b])
        at = P + L - m + np.arange(m)
        lo = np.zeros(m, int) if begin is None else np.maximum(begin[b][:m], 0)
        hi = np.minimum(at + 1 if end is None else end[b][:m], P + L)
        slots = np.arange(P + L)
        seen = (slots >= lo[:, None]) & (slots < hi[:, None])
        use = seen.any(0)
        for hq in range(Hq):
            h = hq // G
            kk, vv = np.concatenate([pk[0, h, :P], k[b, h, :L]])[use], np.concatenate([pv[0, h, :P], v[b, h, :L]])[use]
            worst = max(worst, assert_rows(got[b, hq, :m], q[b, hq, :m], kk, vv, seen[:, use], dtype=dtype, out_dtype=out_dtype,
                                           many=G * n * B > 16, joined=True, slope=0.0 if slopes is None else float(slopes[hq]),
                                           distance=None if slopes is None else np.abs(at[:, None] - slots[None, use]),
                                           lse=None if lse is None else lse[b, hq, :m], **kw))
    return worst


def caches(ctx, B, H, P, cap, lens, seed, paged=False):
    pre, pk, pv = make(ctx, 1, H, P + 40, [P], seed=seed + 50, paged=paged)
    own, k, v = make(ctx, B, H, cap, lens, seed=seed, paged=not paged)
    return pre, own, pk, pv, k, v


CASES = [  # B, heads_q, heads_kv, n_q, prefix, lens
    (1, 1, 1, 1, 1, [1]), (2, 1, 1, 1, 64, [1, 65]), (4, 4, 2, 1, 300, [1, 64, 200, 31]), (3, 4, 4, 1, 129, [10, 0, 700]),
    (2, 16, 2, 1, 700, [100, 900]), (5, 16, 2, 1, 333, [1, 50, 64, 65, 300]), (2, 8, 2, 5, 200, [5, 90]), (40, 8, 2, 1, 500, [1 + 5 * i for i in range(40)]),
    (3, 4, 1, 7, 1000, [7, 100, 64]), (2, 8, 2, 40, 300, [40, 333]), (1, 8, 2, 100, 200, [150]), (3, 4, 2, 129, 100, [129, 200, 300]),
    (70, 4, 1, 1, 4000, [3] * 70), (1, 4, 1, 1, 20000, [9]), (16, 1, 1, 1, 5000, list(range(1, 17))), (2, 6, 1, 50, 64, [20, 50]),
    # rows that fill units of their own: one pass over both caches
    (3, 8, 2, 64, 300, [64, 100, 130]), (2, 4, 1, 32, 1000, [32, 333]), (2, 4, 4, 256, 65, [256, 300]), (1, 8, 1, 250, 129, [700]),
    # too many rows for clusters of few: the kernel for many over the prefix, and over the own tokens
    (64, 64, 8, 1, 300, [5 + b for b in range(64)]), (8, 8, 2, 40, 300, [40 + 30 * b for b in range(8)]), (5, 32, 8, 9, 700, [9, 100, 64, 333, 20]),
    # more sequences and heads than processors: warpgroups with units of their own
    (80, 8, 2, 1, 200, [1 + 3 * i for i in range(80)]), (40, 4, 4, 1, 64, [0, 1, 2000] + [30 * i for i in range(37)]), (200, 3, 1, 1, 100, list(range(200))),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])) + f"-{max(c[5])}")
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, HF), (F32, F32), (BF, F32)])
def test_shared_prefix(ctx, case, dtype, out):
    B, Hq, H, n, P, lens = case
    cap = max(max(lens), n) + 70
    pre, own, pk, pv, k, v = caches(ctx, B, H, P, cap, lens, sum(lens), paged=sum(lens) % 2 == 1)
    q = queries(5, B, Hq, n, dtype, "tokens" if B % 2 else "heads")
    r = np.random.default_rng(P)
    prefix = [P] * B if B % 2 else [P] + r.integers(0, P + 1, B - 1).tolist()
    new = [n] * B
    if n > 1 and B > 1:
        new[-1] = n - 2
    new = [m if L else 0 for m, L in zip(new, lens)]
    lse = torch.empty(B, Hq, n, device=DEV)
    got = torch.full((B, Hq, n, 128), 7.0, dtype=out, device=DEV)
    tq.tq_q8_shared_attention(ctx.handle, pre, ints(prefix), P, own, q, ints(lens), cap, new_lens=ints(new), lse=lse, out=got)
    check(np64(got), np64(q), pk, pv, k, v, prefix, lens, new, dtype=dtype, out_dtype=out, lse=np64(lse))
    for b in range(B):
        assert (got[b, :, new[b]:] == 7.0).all()


@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("B,n", [(2, 1), (9, 2), (2, 60)])
def test_masks_caps_and_biases(ctx, B, n, dtype, out):
    Hq, H, P = 8, 2, 500
    lens = [600 - 50 * b for b in range(B)]
    pre, own, pk, pv, k, v = caches(ctx, B, H, P, 640, lens, 7)
    q = queries(5, B, Hq, n, dtype)
    r = np.random.default_rng(n)
    prefix = r.integers(0, P + 1, B)
    begin, end = r.integers(-50, 900, (B, n)), r.integers(-5, 1300, (B, n))
    begin[0, 0], end[0, 0] = 5, 5
    begin[1, 0], end[1, 0] = -2 ** 31, 2 ** 31 - 1
    slopes = torch.exp2(-torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32))
    for kw, ref in ((dict(key_begin=ints(begin), key_end=ints(end)), dict(begin=begin, end=end)),
                    (dict(key_begin=ints(begin)), dict(begin=begin)),
                    (dict(softcap=20.0, scale=0.2), dict(softcap=20.0, scale=0.2)), (dict(slopes=slopes), dict(slopes=slopes)),
                    (dict(slopes=slopes, softcap=30.0, key_end=ints(end)), dict(slopes=slopes, softcap=30.0, end=end))):
        lse = torch.empty(B, Hq, n, device=DEV)
        got = tq.tq_q8_shared_attention(ctx.handle, pre, ints(prefix), P, own, q, ints(lens), 640, lse=lse, out_dtype=out, **kw)
        check(np64(got), np64(q), pk, pv, k, v, prefix, lens, [n] * B, dtype=dtype, out_dtype=out, lse=np64(lse), **ref)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("n", [1, 60])
def test_heavy_keys_on_either_side(ctx, dtype, n):
    """A row's weight lies in the prefix or in its own tokens by factors of e^60."""
    B, Hq, H, P, lens = 3, 4, 2, 200, [100, 90, 128]
    pre, own, pk, pv, k, v = caches(ctx, B, H, P, 128, lens, 7)
    q = queries(5, B, Hq, n, dtype) * 8
    got = tq.tq_q8_shared_attention(ctx.handle, pre, ints([P] * B), P, own, q, ints(lens), 128)
    check(np64(got), np64(q), pk, pv, k, v, [P] * B, lens, [n] * B, dtype=dtype, out_dtype=dtype)


@pytest.mark.parametrize("n", [1, 20])
def test_queries_that_are_not_finite_stay_alone(ctx, n):
    B, Hq, H, P, lens = 3, 4, 2, 200, [100, 90, 128]
    pre, own, *_ = caches(ctx, B, H, P, 128, lens, 7)
    q = queries(5, B, Hq, n, BF)
    good = tq.tq_q8_shared_attention(ctx.handle, pre, ints([P] * B), P, own, q, ints(lens), 128)
    bad = q.clone()
    bad[1, 2, n - 1, 7] = float("nan")
    got = tq.tq_q8_shared_attention(ctx.handle, pre, ints([P] * B), P, own, bad, ints(lens), 128)
    assert got[1, 2, n - 1].isnan().all()
    got[1, 2, n - 1] = good[1, 2, n - 1]
    assert torch.equal(got, good)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("B,n", [(1, 1), (3, 1), (60, 1), (3, 60), (2, 64), (70, 2)])
def test_either_part_without_tokens(ctx, B, n, dtype):
    """No prefix in any sequence; no own tokens (the queries are the prefix's last tokens, or lie before its first); neither."""
    Hq, H, P, length = 8, 2, 200, 90
    pre, own, pk, pv, k, v = caches(ctx, B, H, P, 128, [length] * B, 7)
    q = queries(5, B, Hq, n, dtype)
    for prefix, have in ((0, length), (P, 0), (30, 0), (0, 0)):
        lse = torch.empty(B, Hq, n, device=DEV)
        got = tq.tq_q8_shared_attention(ctx.handle, pre, ints([prefix] * B), P, own, q, ints([have] * B), 128, lse=lse)
        check(np64(got), np64(q), pk, pv, k, v, [prefix] * B, [have] * B, [n] * B, dtype=dtype, out_dtype=dtype, lse=np64(lse))
        if prefix + have == 0:
            assert not got.any() and torch.isneginf(lse).all()


def test_lengths_and_table_entries_out_of_range(ctx):
    B, Hq, H, P, lens = 3, 4, 2, 200, [100, 90, 128]
    pre, own, pk, pv, k, v = caches(ctx, B, H, P, 128, lens, 7, paged=True)
    for n in (1, 30):
        q = queries(5, B, Hq, n, HF)
        got = tq.tq_q8_shared_attention(ctx.handle, pre, ints([250, -3, P]), P, own, q, ints(lens), 128)
        assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
        check(np64(got), np64(q), pk, pv, k, v, [P, 0, P], lens, [n] * B, dtype=HF, out_dtype=HF)
        was = pre.block_table.clone()
        pre.block_table[:, :, -1] = -1  # (200 tokens: the last of four blocks is not reached by 192 of them)
        got = tq.tq_q8_shared_attention(ctx.handle, pre, ints([192] * B), P, own, q, ints(lens), 128)
        assert tq.tq_get_device_error(ctx.handle) == 0
        check(np64(got), np64(q), pk, pv, k, v, [192] * B, lens, [n] * B, dtype=HF, out_dtype=HF)
        got = tq.tq_q8_shared_attention(ctx.handle, pre, ints([P] * B), P, own, q, ints(lens), 128)
        assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG  # its tokens are taken as unseen
        pre.block_table.copy_(was)


def test_a_batch_served_behind_a_prefix(ctx):
    """Steps of append and attention as one graph, replayed, against eager calls byte for byte; the workspace is one of a larger batch."""
    B, H, Hq, P, cap = 5, 2, 8, 900, 256
    pk, pv = (torch.randn(1, H, P, 128, generator=gen(1 + i), device=DEV).to(BF) for i in range(2))

    def run(graph):
        pre, own = tq.Cache(ctx, 1, H, P), tq.Cache(ctx, B, H, cap)
        tq.tq_q8_append(ctx.handle, pre, pk, pv, ints([0]))
        lens, after, prefix = ints([0, 3, 60, 64, 100]), ints([0] * B), ints([P] * B)
        first = [torch.randn(B, H, 100, 128, generator=gen(5 + i), device=DEV).to(BF) for i in range(2)]
        tq.tq_q8_append(ctx.handle, own, *first, ints([0] * B), new_lens=lens)
        q, nk, nv = (torch.zeros(B, x, 1, 128, dtype=BF, device=DEV) for x in (Hq, H, H))
        out = torch.empty_like(q)
        ws = torch.empty(tq.tq_q8_shared_attention_workspace(ctx.handle, B + 3, Hq, H, 2, 2 * P, 2 * cap), dtype=torch.uint8, device=DEV)

        def step():
            tq.tq_q8_append(ctx.handle, own, nk, nv, lens)
            torch.add(lens, 1, out=after)
            tq.tq_q8_shared_attention(ctx.handle, pre, prefix, P, own, q, after, cap, workspace=ws, out=out)
            lens.copy_(after)

        g, res = None, []
        for i in range(70):
            for t, s in ((q, 10), (nk, 11), (nv, 12)):
                t.copy_(torch.randn(t.shape, generator=gen(100 * i + s), device=DEV).to(BF))
            if graph and g is None:
                was = lens.clone()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step()
                lens.copy_(was)
            g.replay() if graph else step()
            res.append(out.clone())
        return res, [np64(x) for x in (*tq.tq_dequantize(ctx.handle, pre, 0, P), *tq.tq_dequantize(ctx.handle, own, 0, cap))], lens.tolist(), np64(q)

    eager, values, lens, q = run(False)
    for a, b in zip(eager, run(True)[0]):
        assert torch.equal(a, b)
    check(np64(eager[-1]), q, *values, [P] * B, lens, [1] * B, dtype=BF, out_dtype=BF)


def test_replayed_many_times(ctx):
    """A batch of short sequences, thousands of times: the same bytes, and no wait that ran out."""
    B, H, Hq, P = 100, 4, 16, 300
    lens = np.random.default_rng(1).integers(1, 600, B).tolist()
    pre, own, *_ = caches(ctx, B, H, P, 600, lens, 7)
    q, n, p = queries(5, B, Hq, 1, BF), ints(lens), ints([P] * B)
    ws = torch.empty(tq.tq_q8_shared_attention_workspace(ctx.handle, B, Hq, H, 1, P, 600), dtype=torch.uint8, device=DEV)
    first = tq.tq_q8_shared_attention(ctx.handle, pre, p, P, own, q, n, 600)
    outs = [torch.empty_like(q) for _ in range(20)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for out in outs:
            tq.tq_q8_shared_attention(ctx.handle, pre, p, P, own, q, n, 600, workspace=ws, out=out)
    for _ in range(100):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first, out) for out in outs) and tq.tq_get_device_error(ctx.handle) == 0


def test_two_streams(ctx):
    B, Hq, H, P, lens = 3, 8, 2, 200, [100, 90, 128]
    pre, own, pk, pv, k, v = caches(ctx, B, H, P, 128, lens, 7)
    n, p = ints(lens), ints([P] * B)
    qs = [queries(s, B, Hq, 1, HF) for s in (5, 6)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in qs], [None, None]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i] = tq.tq_q8_shared_attention(ctx.handle, pre, p, P, own, qs[i], n, 128, stream=s)
    torch.cuda.synchronize()
    for q, got in zip(qs, outs):
        check(np64(got), np64(q), pk, pv, k, v, [P] * B, lens, [1] * B, dtype=HF, out_dtype=HF)
