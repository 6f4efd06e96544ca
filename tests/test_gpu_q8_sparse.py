"""Attention over listed blocks of the 8-bit cache on the GPU, against fp64 attention over the values that the listed blocks' codes
stand for (oracle/q8_blocks.py), within the bound of tests/q8_rows.py."""

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


def some_lists(B, H, L, n_blocks, lens, seed, nblk):
    """Ascending lists of some of the sequences' blocks (and now and then of one past their end), of any length."""
    r = np.random.default_rng(seed)
    out = np.full((B, H, L, n_blocks), -1, dtype=np.int32)
    for b in range(B):
        have = min(nblk, -(-int(lens[b]) // 64) + 1)
        for h in range(H):
            for l in range(L):
                k = min(have, n_blocks) if r.random() < 0.5 else int(r.integers(0, min(have, n_blocks) + 1))
                out[b, h, l, :k] = np.sort(r.choice(have, k, replace=False))
    return out


def check(got, q, k, v, lists, span, lens, new, *, dtype, out_dtype, begin=None, end=None, slopes=None, q_pos=None, k_pos=None, lse=None, **kw):
    B, Hq, n, _ = q.shape
    H = k.shape[1]
    G = Hq // H
    many = G * min(span, n) > 16
    slots = np.arange(k.shape[2])
    worst = 0.0
    for b in range(B):
        L, m = int(lens[b]), int(new[b])
        at = L - m + np.arange(m)
        lo = np.zeros(m, int) if begin is None else np.maximum(begin[b][:m], 0)
        hi = np.minimum(at + 1 if end is None else end[b][:m], L)
        for hq in range(Hq):
            h = hq // G
            for l in range(-(-m // span)):
                i = slice(l * span, min(m, (l + 1) * span))
                listed = np.isin(slots // 64, lists[b, h, l][lists[b, h, l] >= 0])
                seen = (slots >= lo[i, None]) & (slots < hi[i, None]) & listed
                use = seen.any(0)  # keys that no row sees change nothing (and may be anything)
                dist = None
                if slopes is not None:
                    qp = at[i] if q_pos is None else q_pos[b][:m][i]
                    kp = slots if k_pos is None else k_pos[b, h]
                    dist = np.abs(qp[:, None] - kp[None, use])
                worst = max(worst, assert_rows(got[b, hq, i], q[b, hq, i], k[b, h, use], v[b, h, use], seen[:, use], dtype=dtype, out_dtype=out_dtype,
                                               many=many, slope=0.0 if slopes is None else float(slopes[hq]), distance=dist,
                                               lse=None if lse is None else lse[b, hq, i], **kw))
    return worst


def poison_unlisted(cache, lists):
    """Blocks that no list names are NaN codes."""
    B, H = lists.shape[:2]
    rec = cache.tensors["records"].view(-1, 16384)
    for b in range(B):
        for h in range(H):
            named = set(lists[b, h][lists[b, h] >= 0].tolist())
            for j in range(cache.blocks_per_seq):
                if j not in named:
                    v = (b * H + h) * cache.blocks_per_seq + j
                    rec[v if not isinstance(cache, tq.PagedCache) else int(cache.block_table.view(-1)[v])] = 0x7f


CASES = [  # B, heads_q, heads_kv, n_q, span, n_blocks, lens
    (1, 1, 1, 1, 1, 1, [1]), (1, 1, 1, 1, 1, 3, [130]), (2, 4, 4, 1, 1, 2, [64, 300]), (3, 8, 2, 1, 1, 5, [1000, 65, 64]),
    (2, 12, 4, 1, 1, 9, [1000, 900]), (4, 14, 2, 1, 1, 4, [1, 192, 0, 700]), (2, 32, 2, 1, 1, 7, [2000, 90]), (1, 40, 2, 1, 1, 6, [900]),
    (1, 8, 2, 5, 1, 6, [800]), (2, 4, 4, 5, 5, 3, [5, 930]), (2, 6, 2, 7, 3, 4, [64, 500]), (1, 8, 2, 33, 8, 6, [600]),
    (2, 4, 2, 70, 33, 9, [700, 1100]), (1, 8, 1, 100, 64, 5, [800]), (1, 6, 2, 130, 128, 12, [900]), (2, 2, 1, 150, 200, 8, [900, 150]),
    (40, 2, 2, 1, 1, 3, [1 + 13 * i for i in range(40)]), (1, 4, 1, 1, 1, 300, [20001]), (1, 1, 1, 600, 1, 2, [700]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:6])) + f"-{max(c[6])}")
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, HF), (F32, F32), (HF, F32)])
def test_listed_blocks(ctx, case, dtype, out):
    B, Hq, H, n, span, n_blocks, lens = case
    cap = max(max(lens), n) + 70
    cache, k, v = make(ctx, B, H, cap, lens, seed=sum(lens), paged=sum(lens) % 2 == 1)
    q = queries(5, B, Hq, n, dtype, "tokens" if B % 2 else "heads")
    lists = some_lists(B, H, -(-n // span), n_blocks, lens, sum(lens) + n, cache.blocks_per_seq)
    poison_unlisted(cache, lists)
    new = [min(n, max(0, x)) for x in lens]
    if n > 1 and B > 1:
        new[-1] = min(new[-1], n - 1)
    lse = torch.empty(B, Hq, n, device=DEV)
    got = torch.full((B, Hq, n, 128), 7.0, dtype=out, device=DEV)
    tq.tq_q8_sparse_attention(ctx.handle, cache, torch.from_numpy(lists).to(DEV), q, ints(lens), cap, span=span, new_lens=ints(new), lse=lse, out=got)
    check(np64(got), np64(q), k, v, lists, span, lens, new, dtype=dtype, out_dtype=out, lse=np64(lse))
    for b in range(B):
        assert (got[b, :, new[b]:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("B,Hq,H,longest,n_blocks", [(80, 8, 2, 300, 3), (40, 12, 4, 3000, 40), (160, 1, 1, 700, 9), (600, 3, 1, 130, 2)])
def test_more_lists_than_processors(ctx, B, Hq, H, longest, n_blocks, dtype):
    """Warpgroups with units of their own: short ones, ones that several slices share, sequences without tokens."""
    r = np.random.default_rng(B)
    lens = [longest, 0, 1, 64, 65] + r.integers(0, longest + 1, B - 5).tolist()
    cache, k, v = make(ctx, B, H, longest + 70, lens, seed=B, paged=B % 3 == 0)
    lists = some_lists(B, H, 1, n_blocks, lens, B, cache.blocks_per_seq)
    poison_unlisted(cache, lists)
    q = queries(5, B, Hq, 1, dtype)
    slopes = torch.exp2(-torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32))
    new = r.integers(0, 2, B).tolist()
    new = [min(x, y) for x, y in zip(new, lens)]
    lse = torch.empty(B, Hq, 1, device=DEV)
    for kw, ref in ((dict(), dict()), (dict(softcap=20.0, slopes=slopes, new_lens=ints(new)), dict(softcap=20.0, slopes=slopes))):
        m = new if "new_lens" in kw else [min(1, x) for x in lens]
        got = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
        tq.tq_q8_sparse_attention(ctx.handle, cache, torch.from_numpy(lists).to(DEV), q, ints(lens), longest + 70, lse=lse, out=got, **kw)
        check(np64(got), np64(q), k, v, lists, 1, lens, m, dtype=dtype, out_dtype=dtype, lse=np64(lse), **ref)
        if "new_lens" in kw:
            assert all((got[b] == 7.0).all() for b in range(B) if m[b] == 0)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("Hq,H,n,span,n_blocks,length", [(64, 8, 320, 16, 8, 2000), (4, 1, 2100, 8, 4, 2500), (16, 8, 600, 100, 20, 1500)])
def test_prompts_of_many_lists(ctx, Hq, H, n, span, n_blocks, length, dtype):
    """Slices of whole units, more units than one block plans, units of both sizes."""
    cache, k, v = make(ctx, 1, H, length, [length], seed=n)
    q = queries(5, 1, Hq, n, dtype, "tokens")
    lists = some_lists(1, H, -(-n // span), n_blocks, [length], n, cache.blocks_per_seq)
    got = tq.tq_q8_sparse_attention(ctx.handle, cache, torch.from_numpy(lists).to(DEV), q, ints([length]), length, span=span)
    check(np64(got), np64(q), k, v, lists, span, [length], [n], dtype=dtype, out_dtype=dtype)


def test_replayed_many_times(ctx):
    """Short units one after the other, thousands of times: the same bytes, and no wait that ran out."""
    B, H, Hq = 128, 4, 16
    lens = np.random.default_rng(1).integers(1, 900, B).tolist()
    cache, _, _ = make(ctx, B, H, 900, lens, seed=2)
    lists = torch.from_numpy(some_lists(B, H, 1, 6, lens, 3, cache.blocks_per_seq)).to(DEV)
    q, n = queries(5, B, Hq, 1, BF), ints(lens)
    ws = torch.empty(tq.tq_q8_sparse_attention_workspace(ctx.handle, B, Hq, H, 1, 1, 6), dtype=torch.uint8, device=DEV)
    first = tq.tq_q8_sparse_attention(ctx.handle, cache, lists, q, n, 900)
    outs = [torch.empty_like(q) for _ in range(20)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for out in outs:
            tq.tq_q8_sparse_attention(ctx.handle, cache, lists, q, n, 900, workspace=ws, out=out)
    for _ in range(100):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first, out) for out in outs) and tq.tq_get_device_error(ctx.handle) == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,span", [(3, 1), (100, 64), (300, 128)])
def test_masks_caps_and_biases(ctx, n, span, dtype):
    B, Hq, H, lens = 2, 8, 2, [1500, 777]
    cache, k, v = make(ctx, B, H, 1600, lens, seed=3)
    q = queries(5, B, Hq, n, dtype)
    L = -(-n // span)
    r = np.random.default_rng(n)
    begin, end = r.integers(-50, 1200, (B, n)), r.integers(-5, 2000, (B, n))
    begin[0, :2], end[0, :2] = 5, 5
    slopes = torch.exp2(-torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32))
    q_pos, k_pos = r.integers(0, 3000, (B, n)), r.integers(0, 3000, (B, H, 1600))
    lists = some_lists(B, H, L, 10, lens, n, cache.blocks_per_seq)
    t = torch.from_numpy(lists).to(DEV)
    for kw, ref in ((dict(key_begin=ints(begin), key_end=ints(end)), dict(begin=begin, end=end)),
                    (dict(softcap=20.0), dict(softcap=20.0)), (dict(softcap=500.0, scale=0.3), dict(softcap=500.0, scale=0.3)),
                    (dict(slopes=slopes), dict(slopes=slopes)),
                    (dict(slopes=slopes, q_positions=ints(q_pos), k_positions=ints(k_pos), softcap=30.0),
                     dict(slopes=slopes, q_pos=q_pos, k_pos=k_pos, softcap=30.0))):
        got = tq.tq_q8_sparse_attention(ctx.handle, cache, t, q, ints(lens), 1600, span=span, **kw)
        check(np64(got), np64(q), k, v, lists, span, lens, [n, n], dtype=dtype, out_dtype=dtype, **ref)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("Hq,n", [(4, 1), (16, 1), (8, 3), (8, 40), (8, 200)])
def test_a_list_of_all_blocks_is_the_whole_cache(ctx, Hq, n, dtype):
    """The same attention as over the whole cache: both within one bound of it (their sums are split differently)."""
    lens = [1500]
    cache, k, v = make(ctx, 1, 2, 1536, lens, seed=3)
    q = queries(5, 1, Hq, n, dtype)
    lists = torch.arange(24, dtype=torch.int32, device=DEV).expand(1, 2, 1, 24).contiguous()
    for got in (tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), 1536),
                tq.tq_q8_sparse_attention(ctx.handle, cache, lists, q, ints(lens), 1536, span=n)):
        check(np64(got), np64(q), k, v, lists.cpu().numpy(), n, lens, [n], dtype=dtype, out_dtype=dtype)


def test_bad_lists(ctx):
    cache, k, v = make(ctx, 1, 1, 640, [640], seed=3)
    for n in (1, 40):
        q = queries(5, 1, 1, n, BF)
        good = torch.tensor([1, 4, 9, -1, -1, -1], dtype=torch.int32, device=DEV).view(1, 1, 1, 6)
        want = tq.tq_q8_sparse_attention(ctx.handle, cache, good, q, ints([640]), 640, span=n)
        assert tq.tq_get_device_error(ctx.handle) == 0
        for bad in ([1, 1, 4, 9, -1, -1], [1, 4, 9, 4, -1, -1], [1, 4, 9, 10, -1, -1], [1, 4, 9, -1, 5, -1], [1, 4, 9, 2 ** 31 - 1, -5, -1],
                    [1, 4, 9, -1, 2 ** 31 - 1, 7]):
            t = torch.tensor(bad, dtype=torch.int32, device=DEV).view(1, 1, 1, 6)
            got = tq.tq_q8_sparse_attention(ctx.handle, cache, t, q, ints([640]), 640, span=n)
            assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG, bad
            torch.testing.assert_close(got, want, rtol=2.0 ** -6, atol=2.0 ** -6)
        # negative numbers alone, of any size
        for none in ([-1] * 6, [-2 ** 31] * 6):
            t = torch.tensor(none, dtype=torch.int32, device=DEV).view(1, 1, 1, 6)
            lse = torch.zeros(1, 1, n, device=DEV)
            assert not tq.tq_q8_sparse_attention(ctx.handle, cache, t, q, ints([640]), 640, span=n, lse=lse).any()
            assert torch.isneginf(lse).all() and tq.tq_get_device_error(ctx.handle) == 0


def test_bad_table_entries_and_lengths(ctx):
    cache, k, v = make(ctx, 1, 1, 640, [640], seed=3, paged=True)
    lists = np.array([[[[0, 3, 5, 8]]]], dtype=np.int32)
    for n in (1, 40):
        q = queries(5, 1, 1, n, HF)
        t = torch.from_numpy(lists).to(DEV)
        keep = cache.block_table.clone()
        cache.block_table[0, 0, 3] = cache.pool_blocks
        got = tq.tq_q8_sparse_attention(ctx.handle, cache, t, q, ints([640]), 640, span=n)
        assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
        check(np64(got), np64(q), k, v, np.array([[[[0, 5, 8]]]]), n, [640], [n], dtype=HF, out_dtype=HF)
        cache.block_table.copy_(keep)
        cache.block_table[0, 0, 4] = -1  # not listed: nothing reads it
        got = tq.tq_q8_sparse_attention(ctx.handle, cache, t, q, ints([700]), 640, span=n)
        assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG  # the length, cut
        check(np64(got), np64(q), k, v, lists, n, [640], [n], dtype=HF, out_dtype=HF)
        cache.block_table.copy_(keep)


def test_served_from_prompt_to_decode(ctx):
    """A prompt written, its bounds kept, then steps of append, bounds, choice and attention, captured as one graph and replayed;
    against the same steps over the blocks that the choice names, and eager calls byte for byte."""
    B, H, Hq, cap, prompt, keep = 2, 2, 8, 1280, 900, 6

    def run(graph):
        cache = tq.Cache(ctx, B, H, cap)
        bounds = cache.new_bounds()
        lens = ints([0] * B)
        k, v = (torch.randn(B, H, prompt, 128, generator=gen(1 + i), device=DEV).to(BF) for i in range(2))
        tq.tq_q8_append(ctx.handle, cache, k, v, lens)
        tq.tq_q8_bounds(ctx.handle, cache, bounds, lens, prompt)
        lens += prompt
        ws = torch.empty(max(tq.tq_q8_sparse_attention_workspace(ctx.handle, B, Hq, H, 1, 1, keep), 16), dtype=torch.uint8, device=DEV)
        q, nk, nv = (torch.zeros(B, x, 1, 128, dtype=BF, device=DEV) for x in (Hq, H, H))
        blocks, out = torch.empty(B, H, 1, keep, dtype=torch.int32, device=DEV), torch.empty_like(q)
        after = torch.empty_like(lens)

        def step():
            tq.tq_q8_append(ctx.handle, cache, nk, nv, lens)
            tq.tq_q8_bounds(ctx.handle, cache, bounds, lens, 1)
            torch.add(lens, 1, out=after)
            tq.tq_q8_select(ctx.handle, cache, bounds, q, after, cap, keep, sink=1, recent=2, blocks=blocks)
            tq.tq_q8_sparse_attention(ctx.handle, cache, blocks, q, after, cap, workspace=ws, out=out)
            lens.copy_(after)

        g = None
        res = []
        for i in range(130):
            for t, s in ((q, 10), (nk, 11), (nv, 12)):
                t.copy_(torch.randn(t.shape, generator=gen(100 * i + s), device=DEV).to(BF))
            if not graph:
                step()
            else:
                if g is None:
                    was = lens.clone()
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g):
                        step()
                    lens.copy_(was)
                g.replay()
            res.append((blocks.clone(), out.clone()))
        kv, vv = tq.tq_dequantize(ctx.handle, cache, 0, cap)
        return res, np64(kv), np64(vv), lens.tolist(), np64(q)

    eager, k, v, lens, q = run(False)
    graph = run(True)[0]
    for (b0, o0), (b1, o1) in zip(eager, graph):
        assert torch.equal(b0, b1) and torch.equal(o0, o1)
    assert lens == [prompt + 130] * B
    blocks, out = eager[-1]
    assert (blocks[..., 0] == 0).all() and (blocks[..., -1] == (lens[0] - 1) // 64).all()
    check(np64(out), q, k, v, blocks.cpu().numpy(), 1, lens, [1, 1], dtype=BF, out_dtype=BF)


def test_an_evicted_cache_is_served_on(ctx):
    """A cache cut to its heavy tokens, the bounds of what is left made anew, then a choice among its blocks and attention over them."""
    B, H, Hq, cap, keep_tokens = 2, 2, 8, 1000, 400
    src, _, _ = make(ctx, B, H, cap, [1000, 130], seed=4)
    weights = torch.rand(B, H, cap, generator=gen(3), device=DEV)
    dst = tq.Cache(ctx, B, H, keep_tokens)
    kept, lens, *_ = tq.tq_q8_evict(ctx.handle, src, dst, ints([1000, 130]), weights, keep_tokens)
    assert lens.tolist() == [400, 130]
    bounds = tq.tq_q8_bounds(ctx.handle, dst, dst.new_bounds(), ints([0, 0]), keep_tokens, lens)
    k, v = (np64(x) for x in tq.tq_dequantize(ctx.handle, dst, 0, keep_tokens))
    q = queries(5, B, Hq, 1, BF)
    blocks = tq.tq_q8_select(ctx.handle, dst, bounds, q, lens, keep_tokens, 3, sink=1)
    lists = blocks.cpu().numpy()
    assert (lists[0] >= 0).all() and (lists[0, :, 0, 0] == 0).all() and (lists[0, :, 0, 2] == 6).all() and (lists[1] == [0, 1, 2]).all()
    got = tq.tq_q8_sparse_attention(ctx.handle, dst, blocks, q, lens, keep_tokens)
    check(np64(got), np64(q), k, v, lists, 1, [400, 130], [1, 1], dtype=BF, out_dtype=BF)


def test_two_streams_and_outputs_made_by_the_call(ctx):
    cache, k, v = make(ctx, 2, 2, 640, [640, 500], seed=3)
    lists = some_lists(2, 2, 1, 5, [640, 500], 1, 10)
    t, lens = torch.from_numpy(lists).to(DEV), ints([640, 500])
    qs = [queries(s, 2, 8, 1, HF) for s in (5, 6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [None, None]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i] = tq.tq_q8_sparse_attention(ctx.handle, cache, t, qs[i], lens, 640, stream=s)
    torch.cuda.synchronize()
    for q, got in zip(qs, outs):
        check(np64(got), np64(q), k, v, lists, 1, [640, 500], [1, 1], dtype=HF, out_dtype=HF)
