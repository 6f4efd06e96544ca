"""Key bounds of blocks and the choice of blocks on the GPU: whole numbers, equal to the oracle's (oracle/q8_blocks.py)."""

import numpy as np
import pytest
import torch

from oracle import q8_blocks as ob
from quantised_kv_cache_gb300 import tq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


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
    c.close()


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def error(ctx):
    return tq.tq_get_device_error(ctx.handle)


def make_cache(ctx, B, H, cap, paged=False, seed=0, records=True, exponents=(-9, -4)):
    """Random finite codes and scales; the pool's blocks in a random order, with some to spare."""
    r = np.random.default_rng(seed)
    nblk = -(-cap // 64)
    n = B * H * nblk
    if paged:
        table = torch.from_numpy(r.permutation(n + 3)[:n].astype(np.int32)).view(B, H, nblk).to(DEV)
        cache = tq.PagedCache(ctx, B, H, cap, n + 3, table)
    else:
        cache = tq.Cache(ctx, B, H, cap)
    if records:
        rec = torch.from_numpy(r.integers(0, 256, cache.tensors["records"].numel(), dtype=np.uint8))
        rec[(rec & 0x7f) == 0x7f] = 0x80
        # blocks whose codes all have one sign, or are all zeros of one sign, in some coordinates
        keys = rec.view(-1, 2, 8192)[:, 0].view(-1, 8, 8, 8, 16)  # [block][group][column][token][16]
        keys[..., 0] |= 0x80
        keys[..., 1] &= 0x7f
        keys[..., 2] = 0x80
        keys[..., 3] = 0
        cache.tensors["records"].copy_(rec)
    e = r.integers(exponents[0], exponents[1] + 1, cache.bounds_blocks)
    cache.tensors["k_stats"].view(F32).copy_(torch.from_numpy(np.ldexp(1.0, e).astype(np.float32)))
    return cache, e


def physical(cache, b, h, j):
    v = (b * cache.heads_kv + h) * cache.blocks_per_seq + j
    return v if not isinstance(cache, tq.PagedCache) else int(cache.block_table.view(-1)[v])


def key_codes(cache):
    """float64 [blocks][64][128] of all blocks as they lie."""
    plane = cache.tensors["records"].view(-1, 2, 8192)[:, 0].reshape(-1, 8, 8, 8, 16).transpose(2, 3).reshape(-1, 64, 128)
    return plane.view(torch.float8_e4m3fn).double().cpu().numpy()


# ------------------------------------------------------------------------------------------------ bounds

@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,H,cap,n,lens,new", [
    (1, 1, 64, 1, [0], None), (1, 1, 64, 1, [63], None), (2, 3, 200, 1, [64, 130], None), (3, 2, 500, 2, [63, 0, 127], None),
    (4, 2, 700, 65, [63, 1, 64, 500], [65, 0, 1, 64]), (1, 5, 1000, 1000, [0], None), (2, 1, 1000, 300, [700, 5], [300, 299]),
    (40, 1, 130, 66, list(range(0, 63, 2)) + [63] * 8, None),
])
def test_bounds(ctx, B, H, cap, n, lens, new, paged):
    cache, _ = make_cache(ctx, B, H, cap, paged, seed=B + n)
    bounds = cache.new_bounds().fill_(77)
    got = tq.tq_q8_bounds(ctx.handle, cache, bounds, ints(lens), n, None if new is None else ints(new))
    assert got is bounds
    want = np.full((cache.bounds_blocks, 2, 128), 77)
    codes = key_codes(cache)
    for b in range(B):
        m = n if new is None else new[b]
        for j in range(lens[b] // 64, -(-(lens[b] + m) // 64) if m else 0):
            for h in range(H):
                at = physical(cache, b, h, j)
                want[at] = ob.bounds(codes[at, :lens[b] + m - 64 * j])
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert error(ctx) == 0


def test_bounds_cover_every_code(ctx):
    """Each e4m3 number alone in its coordinate: floor and ceiling of its quarter."""
    cache = tq.Cache(ctx, 1, 1, 128)
    codes = np.array([c for c in range(256) if c & 0x7f != 0x7f] + [0x80] * 2, dtype=np.uint8).reshape(2, 128)
    rec = np.zeros((2, 2, 8192), dtype=np.uint8)
    for j in range(2):
        for c in range(128):
            rec[j, 0, 128 * (c // 16) + c % 16] = codes[j, c]  # token 0
    cache.tensors["records"].copy_(torch.from_numpy(rec).view(-1))
    got = tq.tq_q8_bounds(ctx.handle, cache, cache.new_bounds(), ints([0]), 1)[0].cpu().numpy()
    value = torch.from_numpy(codes[0]).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(got, np.stack([np.floor(value / 4), np.ceil(value / 4)]))
    got = tq.tq_q8_bounds(ctx.handle, cache, cache.new_bounds(), ints([64]), 1)[1].cpu().numpy()
    value = torch.from_numpy(codes[1]).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(got, np.stack([np.floor(value / 4), np.ceil(value / 4)]))


def test_bounds_of_sequences_that_do_not_fit(ctx):
    cache, _ = make_cache(ctx, 3, 2, 128)
    bounds = cache.new_bounds()
    tq.tq_q8_bounds(ctx.handle, cache, bounds, ints([126, -1, 0]), 3)
    assert error(ctx) == tq.TQ_ERR_CAPACITY
    got = bounds.view(3, 2, 2, 256).cpu().numpy()
    assert not got[:2].any() and got[2, :, 0].any() and not got[2, :, 1].any()
    bounds.zero_()
    tq.tq_q8_bounds(ctx.handle, cache, bounds, ints([0, 0, 0]), 3, ints([4, -1, 0]))
    assert error(ctx) == tq.TQ_ERR_ARG and not bounds.any()
    # a call that could bring more tokens than there are slots
    tq.tq_q8_bounds(ctx.handle, cache, bounds, ints([100, 0, 0]), 2 ** 31 - 1, ints([28, 0, 0]))
    assert error(ctx) == 0 and bounds.view(3, -1)[0].any() and not bounds.view(3, -1)[1:].any()


def test_bounds_of_a_bad_table_entry(ctx):
    cache, _ = make_cache(ctx, 1, 2, 128, paged=True)
    cache.block_table[0, 1, 1] = cache.pool_blocks
    bounds = cache.new_bounds()
    tq.tq_q8_bounds(ctx.handle, cache, bounds, ints([0]), 128)
    assert error(ctx) == tq.TQ_ERR_ARG
    there = {physical(cache, 0, h, j) for h, j in ((0, 0), (0, 1), (1, 0))}
    assert [bool(x.any()) for x in bounds] == [i in there for i in range(cache.pool_blocks)]


def test_bounds_after_appends_that_raise_the_scale(ctx):
    """A block's older codes are rounded again when its scale grows: the bounds follow."""
    cache = tq.Cache(ctx, 1, 1, 64)
    bounds = cache.new_bounds()
    g = torch.Generator(device=DEV).manual_seed(3)
    for t in range(20):
        x = torch.randn(1, 1, 1, 128, generator=g, device=DEV) * 1.7 ** t
        tq.tq_q8_append(ctx.handle, cache, x, x, ints([t]))
        tq.tq_q8_bounds(ctx.handle, cache, bounds, ints([t]), 1)
        np.testing.assert_array_equal(bounds[0].cpu().numpy(), np.stack(ob.bounds(key_codes(cache)[0, :t + 1])))


# ------------------------------------------------------------------------------------------------ the choice

def some_bounds(cache, seed):
    r = np.random.default_rng(seed)
    x = np.sort(r.integers(-112, 113, (cache.bounds_blocks, 2, 128)), axis=1)
    return torch.from_numpy(x.astype(np.int8)).to(DEV)


def want_lists(cache, e, bounds, q, lens, new, span, keep, sink, recent, begin=None, end=None):
    B, Hq, n, _ = q.shape
    H = cache.heads_kv
    G, L = Hq // H, -(-n // span)
    q = q.double().cpu().numpy()
    bounds = bounds.cpu().numpy()
    out = np.full((B, H, L, keep), -1)
    for b in range(B):
        m = n if new is None else new[b]
        at = lens[b] - m + np.arange(m)
        lo = np.zeros(m, int) if begin is None else np.maximum(begin[b][:m], 0)
        hi = np.minimum(at + 1 if end is None else end[b][:m], lens[b])
        for l in range(L):
            rows = [i for i in range(l * span, min(m, (l + 1) * span)) if hi[i] > lo[i]]
            if not rows:
                continue
            first, last = min(lo[i] for i in rows) // 64, -(-max(hi[i] for i in rows) // 64)
            for h in range(H):
                p = [physical(cache, b, h, j) for j in range(first, last)]
                s = ob.scores(q[b, h * G:(h + 1) * G][:, rows].reshape(-1, 128), bounds[p, 0], bounds[p, 1], e[p])
                got = ob.choose(s, first, last, keep, sink, recent)
                out[b, h, l, :len(got)] = got
    return out


def queries(B, Hq, n, dtype, seed=0, layout="heads"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(B, Hq, n, 128, generator=g, device=DEV) * torch.exp(torch.randn(B, Hq, 1, 1, generator=g, device=DEV))
    return x.transpose(1, 2).contiguous().to(dtype).transpose(1, 2) if layout == "tokens" else x.to(dtype)


CASES = [  # B, heads_q, heads_kv, n_q, span, lens, keep, sink, recent
    (1, 1, 1, 1, 1, [1], 1, 0, 1), (1, 1, 1, 1, 1, [65], 1, 0, 1), (1, 1, 1, 1, 1, [500], 3, 1, 1), (1, 4, 1, 1, 1, [4000], 10, 0, 0),
    (2, 4, 4, 1, 1, [640, 641], 4, 2, 2), (3, 8, 2, 1, 1, [3000, 0, 1], 5, 1, 1), (1, 16, 1, 1, 1, [10000], 20, 1, 2), (1, 20, 1, 1, 1, [9000], 7, 1, 1),
    (2, 6, 2, 3, 1, [3, 5000], 8, 1, 2), (2, 8, 4, 5, 5, [5, 2000], 6, 0, 1), (2, 4, 2, 33, 8, [700, 2600], 6, 1, 2), (1, 8, 2, 200, 64, [200], 2, 0, 1),
    (1, 8, 2, 130, 64, [3333], 9, 1, 3), (1, 2, 1, 300, 1000, [3000], 5, 1, 1), (40, 2, 1, 1, 1, [64 * i + 1 for i in range(40)], 8, 1, 1),
    (1, 4, 1, 1, 1, [64 * 1000], 64, 1, 2), (1, 1, 1, 1, 1, [64 * 5000 + 7], 100, 1, 2), (1, 16, 8, 1, 1, [64 * 1030], 17, 0, 0),
    (1, 4, 2, 2, 1, [64 * 520], 520, 1, 1),
    # lists of several tiles: a processor's slice is whole lists; begins within one
    (1, 8, 2, 512, 8, [64 * 300], 9, 1, 1), (1, 8, 2, 640, 8, [64 * 300], 9, 1, 1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])) + f"-{max(c[5])}-{c[6]}")
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_choice(ctx, case, dtype):
    B, Hq, H, n, span, lens, keep, sink, recent = case
    cap = max(max(lens), n)
    cache, e = make_cache(ctx, B, H, cap, paged=sum(lens) % 2 == 1, seed=sum(lens), records=False)
    bounds = some_bounds(cache, 5)
    q = queries(B, Hq, n, dtype, layout="tokens" if B % 2 else "heads")
    ragged = n > 1 and B > 1
    new = [n] + [max(0, n - 2 * i) for i in range(1, B)] if ragged else None
    got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints(lens), cap, keep, sink=sink, recent=recent, span=span,
                          new_lens=ints(new) if ragged else None)
    want = want_lists(cache, e, bounds, q, lens, new, span, keep, sink, recent)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert error(ctx) == 0


def test_choice_of_more_blocks_than_shared_memory_holds(ctx):
    lens = [64 * 33000 + 5]
    cache, e = make_cache(ctx, 1, 1, lens[0], seed=3)
    bounds = some_bounds(cache, 6)
    for heads, n, span in ((1, 1, 1), (5, 1, 1), (4, 9, 9)):  # the last in several passes over the rows
        q = queries(1, heads, n, BF, seed=heads)
        got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints(lens), lens[0], 1000, sink=1, recent=2, span=span)
        np.testing.assert_array_equal(got.cpu().numpy(), want_lists(cache, e, bounds, q, lens, None, span, 1000, 1, 2))
    assert error(ctx) == 0


def test_choice_within_key_ranges(ctx):
    B, Hq, H, n, span = 2, 4, 2, 12, 4
    lens = [5000, 2111]
    cache, e = make_cache(ctx, B, H, 5000, seed=8, records=False)
    bounds = some_bounds(cache, 9)
    q = queries(B, Hq, n, BF)
    r = np.random.default_rng(1)
    begin, end = r.integers(-100, 3000, (B, n)), r.integers(-5, 6000, (B, n))
    begin[0, 4:8], end[0, 4:8] = 100, 100  # a list whose rows see nothing
    got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints(lens), 5000, 6, sink=1, recent=1, span=span, key_begin=ints(begin), key_end=ints(end))
    want = want_lists(cache, e, bounds, q, lens, None, span, 6, 1, 1, begin, end)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert (want[0, :, 1] == -1).all() and error(ctx) == 0


@pytest.mark.parametrize("n", [1, 40])
def test_equal_scores_go_to_the_lowest_blocks(ctx, n):
    cache, _ = make_cache(ctx, 1, 1, 64 * 300, records=False, exponents=(0, 0))
    bounds = torch.ones(300, 2, 128, dtype=torch.int8, device=DEV)
    bounds[250:] = 2  # the better ones among the last
    q = torch.ones(1, 1, n, 128, dtype=BF, device=DEV)
    got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints([64 * 300]), 64 * 300, 80, sink=0, recent=0, span=n)
    np.testing.assert_array_equal(got.cpu().numpy().ravel(), [*range(30), *range(250, 300)])


@pytest.mark.parametrize("n", [1, 40])
def test_scores_at_the_ends_of_float32(ctx, n):
    """Scales from 2^-100 to 2^119 and queries from subnormal to 2^127: exact all the same."""
    cache, e = make_cache(ctx, 1, 1, 64 * 200, records=False, exponents=(-100, 119))
    bounds = some_bounds(cache, 2)
    bounds[::7] = 0
    bounds[1::7] = bounds[1::7].clamp(-112, -1)
    for size in (2.0 ** -140, 2.0 ** -120, 1.0, 2.0 ** 127):
        q = (torch.rand(1, 2, n, 128, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) - 0.5) * size
        got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints([64 * 200]), 64 * 200, 50, span=n)
        want = want_lists(cache, e, bounds, q, [64 * 200], None, n, 50, 0, 1)
        np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("n", [1, 40])
def test_rows_that_are_not_finite_do_not_count(ctx, n):
    cache, e = make_cache(ctx, 1, 1, 64 * 100, records=False)
    bounds = some_bounds(cache, 2)
    q = queries(1, 4, n, BF)
    q[0, 1, 0, 5], q[0, 2, n - 1, 7] = float("inf"), float("nan")
    got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints([6400]), 6400, 20, span=n)
    np.testing.assert_array_equal(got.cpu().numpy(), want_lists(cache, e, bounds, q, [6400], None, n, 20, 0, 1))
    q.fill_(float("nan"))
    got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints([6400]), 6400, 20, span=n)
    np.testing.assert_array_equal(got.cpu().numpy().ravel(), [*range(19), 99])


def test_lengths_out_of_range_and_bad_table_entries(ctx):
    cache, e = make_cache(ctx, 2, 1, 640, paged=True, records=False)
    bounds = some_bounds(cache, 2)
    q = queries(2, 1, 1, BF)
    got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints([1000, -5]), 640, 5)
    assert error(ctx) == tq.TQ_ERR_ARG
    want = want_lists(cache, e, bounds, q, [640, 0], None, 1, 5, 0, 1)
    # the query's slot is its length's last; a length cut to 640 leaves it there
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    cache.block_table[0, 0, 2], cache.block_table[0, 0, 5] = -1, cache.pool_blocks
    got = tq.tq_q8_select(ctx.handle, cache, bounds, q, ints([640, 64]), 640, 8)
    assert error(ctx) == tq.TQ_ERR_ARG
    np.testing.assert_array_equal(got.cpu().numpy()[0].ravel(), [0, 1, 3, 4, 6, 7, 8, 9])


def test_no_workspace_state_and_replays(ctx):
    """Captured once, replayed with other inputs in the same buffers; two captures share nothing."""
    cache, e = make_cache(ctx, 2, 2, 6400, records=False)
    bounds, lens = some_bounds(cache, 2), ints([6400, 3000])
    q = queries(2, 8, 1, BF)
    out = torch.empty(2, 2, 1, 12, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tq.tq_q8_select(ctx.handle, cache, bounds, q, lens, 6400, 12, blocks=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_q8_select(ctx.handle, cache, bounds, q, lens, 6400, 12, blocks=out)
    for k in range(3):
        q.copy_(queries(2, 8, 1, BF, seed=20 + k))
        lens.copy_(ints([6400 - 700 * k, 3000 + 64 * k]))
        out.fill_(-7)
        g.replay()
        np.testing.assert_array_equal(out.cpu().numpy(), want_lists(cache, e, bounds, q, lens.tolist(), None, 1, 12, 0, 1))
