"""The 8-bit cache (append, dequantise, eviction) and rotary positions on the GPU against their fp64
restatement (oracle/q8.py). Codes, scales and kept slots are exact; the rotation's tolerance counts its
roundings."""

import numpy as np
import pytest
import torch

from oracle import q8
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


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def randn(seed, *shape, dtype=BF):
    return torch.randn(shape, generator=gen(seed), device=DEV).to(dtype)


def np64(t):
    return t.double().cpu().numpy()


def paged(ctx, B, H, cap, seed=0, spare=3):
    n = B * H * (-(-cap // 64))
    pool = n + spare
    table = torch.from_numpy(np.random.default_rng(seed).permutation(pool)[:n].astype(np.int32)).view(B, H, -1).to(DEV)
    return tq.PagedCache(ctx, B, H, cap, pool, table, device=DEV)


# ------------------------------------------------------------------------------------------------ rotary

# the sine and cosine: 2^-32 turns of angle, 2^-24 rounding of x <= pi/4, two polynomial roundings near 1
SINCOS = 2.0 ** -22


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("dim,interleaved", [(128, False), (128, True), (64, False), (64, True), (72, False), (72, True), (8, False), (8, True)])
def test_rotary_equals_the_formula(ctx, dtype, dim, interleaved):
    B, H, n = 2, 5, 37
    kw = dict(base=500000.0, factor=8.0, original_len=4096.0, low=1.0, high=4.0)
    tq.tq_set_rope(ctx.handle, dim, interleaved, gain=1.2, **kw)
    x = randn(2, B, n, H, 128, dtype=dtype).transpose(1, 2)  # token-major
    pos = torch.randint(-5000, 2 ** 31 - 1, (B, n), generator=gen(3), device=DEV, dtype=torch.int64)
    pos[:, :20] = torch.arange(20, device=DEV)
    pos[0, 20], pos[0, 21] = 2 ** 31 - 1, -2 ** 31
    for transpose in (False, True):
        y = tq.tq_rotary(ctx.handle, x, pos.int(), transpose=transpose)
        assert y.stride() == x.stride()
        want = q8.rope(np64(x), pos.cpu().numpy()[:, None, :], dim, interleaved, gain=1.2, transpose=transpose, **kw)
        # angles of far positions: fp64's own error in the oracle is pos * f * 2^-52 radians
        half = (slice(0, dim, 2), slice(1, dim, 2)) if interleaved else (slice(0, dim // 2), slice(dim // 2, dim))
        size = np.zeros_like(want)
        xa = np.abs(np64(x))
        size[..., half[0]] = size[..., half[1]] = xa[..., half[0]] + xa[..., half[1]]
        tol = 1.2 * size * (SINCOS + 3 * 2.0 ** -24 + 2.0 ** 31 * 2.0 ** -51) + np.abs(want) * torch.finfo(dtype).eps / 2 * 1.01
        got = np64(y)
        assert np.all(np.abs(got - want) <= tol)
        np.testing.assert_array_equal(got[..., dim:], np64(x)[..., dim:])


@pytest.mark.parametrize("B,H,n", [(1, 1, 1), (16, 32, 1), (3, 7, 5), (1, 40, 2000), (2, 32, 4099)])
def test_rotary_sizes_in_place_and_into_another_layout(ctx, B, H, n):
    tq.tq_set_rope(ctx.handle)
    x = randn(4, B, H, n, 128)
    pos = torch.arange(n, dtype=torch.int32, device=DEV) + 11 * torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    want = tq.tq_rotary(ctx.handle, x, pos.contiguous())
    other = torch.full((B, n, H, 136), 7.0, dtype=BF, device=DEV)
    tq.tq_rotary(ctx.handle, x, pos.contiguous(), out=other.transpose(1, 2)[..., :128])
    assert torch.equal(other.transpose(1, 2)[..., :128], want) and bool((other[..., 128:] == 7).all())
    some = np64(want[:, :, -3:]), q8.rope(np64(x[:, :, -3:]), pos.cpu().numpy()[:, None, -3:], 128)
    assert np.max(np.abs(some[0] - some[1])) < 2.0 ** -8 * 8
    tq.tq_rotary(ctx.handle, x, pos.contiguous(), out=x)
    assert torch.equal(x, want)


# ------------------------------------------------------------------------------------------------ append

class Pair:
    """The oracle's model of a cache, keys and values."""

    def __init__(self, B, H, cap):
        self.B, self.H = B, H
        self.k, self.v = q8.Model(B * H, cap), q8.Model(B * H, cap)

    def append(self, lens, k, v, new=None):
        k, v = np64(k), np64(v)
        for b in range(self.B):
            n = k.shape[2] if new is None else int(new[b])
            for h in range(self.H):
                self.k.append(b * self.H + h, int(lens[b]), k[b, h, :n])
                self.v.append(b * self.H + h, int(lens[b]), v[b, h, :n])

    def check(self, ctx, cache, lens):
        n = cache.capacity
        k, v = tq.tq_dequantize(ctx.handle, cache, 0, n)
        for got, model in ((k, self.k), (v, self.v)):
            got = np64(got).reshape(self.B * self.H, n, 128)
            want = model.values()
            for b in range(self.B):
                rows = slice(b * self.H, (b + 1) * self.H)
                np.testing.assert_array_equal(got[rows, :lens[b]], want[rows, :lens[b]])


def spread(seed, *shape, dtype=BF):
    """Vectors whose magnitudes differ widely from token to token."""
    x = torch.randn(shape, generator=gen(seed), device=DEV)
    return (x * torch.exp2(torch.randint(-9, 10, shape[:-1] + (1,), generator=gen(seed + 1), device=DEV).float())).to(dtype)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("layout", ["contiguous", "paged"])
def test_append_codes_equal_the_oracles(ctx, dtype, layout):
    B, H, cap = 3, 4, 300
    cache = tq.Cache(ctx, B, H, cap, device=DEV) if layout == "contiguous" else paged(ctx, B, H, cap)
    model, lens = Pair(B, H, cap), np.array([0, 5, 63])
    first = spread(1, B, H, 63, 128, dtype=dtype), spread(3, B, H, 63, 128, dtype=dtype)
    tq.tq_q8_append(ctx.handle, cache, *first, ints([0, 0, 0]), new_lens=ints(lens))
    model.append([0, 0, 0], *first, new=lens)
    for i, (n, new) in enumerate([(1, None), (1, [1, 0, 1]), (64, None), (3, [3, 1, 2]), (100, [100, 37, 0]), (1, None)]):
        # token-major inputs with rows between that are not read
        k = torch.full((B, n, H + 1, 128), float("nan"), device=DEV, dtype=dtype)
        v = torch.full((B, n, H + 1, 128), float("nan"), device=DEV, dtype=dtype)
        k[:, :, :H], v[:, :, :H] = (spread(10 * i + j, B, n, H, 128, dtype=dtype) for j in (5, 7))
        k, v = k[:, :, :H].transpose(1, 2), v[:, :, :H].transpose(1, 2)
        if new is not None:  # what lies behind a sequence's tokens is not read
            for b in range(B):
                k[b, :, new[b]:], v[b, :, new[b]:] = float("nan"), float("inf")
        tq.tq_q8_append(ctx.handle, cache, k, v, ints(lens), new_lens=None if new is None else ints(new))
        model.append(lens, k, v, new)
        lens = lens + (n if new is None else np.array(new))
        assert tq.tq_get_device_error(ctx.handle) == 0
        model.check(ctx, cache, lens)


def test_token_by_token_and_the_general_call(ctx):
    """tq_append_quantize writes what tq_q8_append writes; single tokens rescale their block as they come."""
    B, H, n = 2, 3, 130
    a, b = tq.Cache(ctx, B, H, 192, device=DEV), tq.Cache(ctx, B, H, 192, device=DEV)
    k, v = spread(1, B, H, n, 128), spread(2, B, H, n, 128)
    model = Pair(B, H, 192)
    for t in range(n):
        at, kt, vt = ints([t, t]), k[:, :, t:t + 1].contiguous(), v[:, :, t:t + 1].contiguous()
        tq.tq_append_quantize(ctx.handle, a, kt, vt, at)
        tq.tq_q8_append(ctx.handle, b, kt, vt, at)
        model.append([t, t], kt, vt)
    for name in a.tensors:
        assert torch.equal(a.tensors[name], b.tensors[name])
    model.check(ctx, a, [n, n])


@pytest.mark.parametrize("x", [0.0, 1e-45, 1e-38, 2.0 ** -92, 1e30, 3.4e38])
def test_extreme_blocks(ctx, x):
    cache = tq.Cache(ctx, 1, 1, 64, device=DEV)
    k = torch.zeros(1, 1, 2, 128, device=DEV)
    k[..., ::3], k[..., 1::3] = x, -x / 3
    model = Pair(1, 1, 64)
    tq.tq_q8_append(ctx.handle, cache, k, -k, ints([0]))
    model.append([0], k, -k)
    model.check(ctx, cache, [2])


def test_numbers_that_are_not_finite(ctx):
    cache = tq.Cache(ctx, 1, 2, 64, device=DEV)
    k = randn(1, 1, 2, 20, 128, dtype=F32)
    k[0, 0, 3, 5], k[0, 1, 4, 6], k[0, 1, 4, 7] = float("inf"), float("nan"), float("-inf")
    v = randn(2, 1, 2, 20, 128, dtype=F32)
    model = Pair(1, 2, 64)
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([0]))
    model.append([0], k, v)
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_NONFINITE
    model.check(ctx, cache, [20])


@pytest.mark.parametrize("dim,interleaved", [(128, False), (128, True), (64, False), (72, False), (72, True), (8, False)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_with_rotation_equals_the_rotary_call_before_it(ctx, dim, interleaved, dtype):
    B, H, n = 2, 11, 70
    tq.tq_set_rope(ctx.handle, dim, interleaved, base=10000.0, factor=4.0, original_len=100.0, low=1.0, high=32.0, gain=1.1)
    k, v = randn(1, B, H, n, 128, dtype=dtype), randn(2, B, H, n, 128, dtype=dtype)
    lens = ints([0, 30])
    for pos in (None, ints(np.arange(2 * n).reshape(2, n) * 1001)):
        a, b = tq.Cache(ctx, B, H, 128, device=DEV), tq.Cache(ctx, B, H, 128, device=DEV)
        tq.tq_q8_append(ctx.handle, a, k, v, lens, rope=True, positions=pos)
        at = pos if pos is not None else (lens[:, None] + torch.arange(n, device=DEV, dtype=torch.int32)).int().contiguous()
        tq.tq_q8_append(ctx.handle, b, tq.tq_rotary(ctx.handle, k, at), v, lens)
        for name in a.tensors:
            assert torch.equal(a.tensors[name], b.tensors[name])


def test_appends_that_do_not_fit_are_skipped_whole(ctx):
    B, H, cap = 4, 2, 100
    cache = tq.Cache(ctx, B, H, cap, device=DEV)
    for t in cache.tensors.values():
        t.fill_(0x11)
    was = cache.tensors["records"].clone()
    k, v = randn(1, B, H, 5, 128), randn(2, B, H, 5, 128)
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([96, -1, 2 ** 31 - 3, 101]))
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_CAPACITY
    assert torch.equal(cache.tensors["records"], was)
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([0, 0, 0, 0]), new_lens=ints([6, -1, 0, 0]))
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    assert torch.equal(cache.tensors["records"], was)
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([95, 0, 0, 0]))
    assert tq.tq_get_device_error(ctx.handle) == 0


def test_bad_table_entries_are_skipped(ctx):
    B, H, cap = 1, 2, 128
    cache = paged(ctx, B, H, cap)
    cache.block_table[0, 0, 1], cache.block_table[0, 1, 0] = -1, cache.pool_blocks
    k, v = randn(1, B, H, 100, 128), randn(2, B, H, 100, 128)
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([0]))
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    model = Pair(B, H, cap)
    model.append([0], k, v)
    got, _ = tq.tq_dequantize(ctx.handle, cache, 0, 128)
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    np.testing.assert_array_equal(np64(got)[0, 0, :64], model.k.values()[0, :64])
    np.testing.assert_array_equal(np64(got)[0, 1, 64:100], model.k.values()[1, 64:100])


# ------------------------------------------------------------------------------------------------ eviction

def fill(ctx, cache, lens, seed):
    B, H = cache.batch, cache.heads_kv
    n = max(int(max(lens)), 1)
    k, v = spread(seed, B, H, n, 128), spread(seed + 1, B, H, n, 128)
    zero = ints([0] * B)
    tq.tq_q8_append(ctx.handle, cache, k, v, zero, new_lens=ints(lens))


def check_evict(ctx, src, dst, lens, w, keep, sink, recent, pos):
    B, H = src.batch, src.heads_kv
    kept, dlens, dw, dp = tq.tq_q8_evict(ctx.handle, src, dst, ints(lens), w, keep, sink, recent, positions=pos)
    ks, vs = (np64(t) for t in tq.tq_dequantize(ctx.handle, src, 0, src.capacity))
    kd, vd = (np64(t) for t in tq.tq_dequantize(ctx.handle, dst, 0, dst.capacity))
    wn, kept, dw, dp = w.cpu().numpy(), kept.cpu().numpy(), dw.cpu().numpy(), dp.cpu().numpy()
    slots = -(-keep // 64) * 64
    for b in range(B):
        n = int(min(max(lens[b], 0), src.capacity))
        m = min(n, keep)
        assert int(dlens[b]) == m
        for h in range(H):
            stay = q8.evict(wn[b, h], n, keep, sink, recent)
            np.testing.assert_array_equal(kept[b, h], np.concatenate([stay, np.full(keep - m, -1)]))
            np.testing.assert_array_equal(dw[b, h], np.concatenate([wn[b, h][stay], np.zeros(dst.capacity - m, np.float32)]))
            want_pos = stay if pos is None else pos.cpu().numpy()[b, h][stay]
            np.testing.assert_array_equal(dp[b, h], np.concatenate([want_pos, np.zeros(dst.capacity - m)]))
            for s, d in ((ks, kd), (vs, vd)):
                model = q8.Model(1, slots)
                x = np.zeros((slots, 128))
                x[:m] = s[b, h][stay]
                model.append(0, 0, x)
                top = min(slots, dst.capacity)
                np.testing.assert_array_equal(d[b, h, :top], model.values()[0, :top])


@pytest.mark.parametrize("cap,lens,keep,sink,recent", [
    (64, [1, 64], 1, 0, 0), (64, [1, 64], 1, 1, 0), (100, [0, 100], 64, 4, 10), (300, [300, 299], 299, 0, 299),
    (1000, [1000, 500], 65, 0, 1), (1000, [999, 64], 500, 13, 487), (8300, [8300, 8191], 1000, 4, 128),
    (40000, [40000, 20001], 4097, 0, 0), (70000, [70000, 65536], 2000, 3, 64)])
@pytest.mark.parametrize("kind", ["heavy", "ties"])
def test_eviction_keeps_the_heaviest(ctx, cap, lens, keep, sink, recent, kind):
    H = 2
    src, dst = tq.Cache(ctx, 2, H, cap, device=DEV), paged(ctx, 2, H, keep + 7)
    fill(ctx, src, lens, 5)
    w = torch.exp(2 * torch.randn(2, H, cap, generator=gen(8), device=DEV))
    if kind == "ties":
        w = (w * 2).floor()
        w[0, 0] = 1.0  # all equal
        w[1, 1, ::7] = float("nan")
        w[1, 0, ::5], w[1, 0, 1::5], w[1, 0, 2::11] = -0.0, float("-inf"), float("inf")
    pos = torch.randint(0, 10 ** 6, (2, H, cap), generator=gen(9), device=DEV, dtype=torch.int32)
    check_evict(ctx, src, dst, lens, w, keep, sink, recent, pos if kind == "heavy" else None)
    assert tq.tq_get_device_error(ctx.handle) == 0


def test_eviction_of_a_ragged_batch(ctx):
    """Sequences on both sides of the budget, again and again into the same target."""
    B, H, cap, keep = 16, 8, 2048, 1000
    src, dst = tq.Cache(ctx, B, H, cap, device=DEV), tq.Cache(ctx, B, H, keep, device=DEV)
    lens = [2048, 1, 999, 1000, 1001, 1500, 64, 0] + [100 * i for i in range(1, 9)]
    fill(ctx, src, lens, 5)
    for i in range(3):
        w = torch.rand(B, H, cap, generator=gen(i), device=DEV)
        first = [t.clone() for t in tq.tq_q8_evict(ctx.handle, src, dst, ints(lens), w, keep, 16, 500)]
        for _ in range(5):
            again = tq.tq_q8_evict(ctx.handle, src, dst, ints(lens), w, keep, 16, 500)
            assert all(torch.equal(x, y) for x, y in zip(first, again))
    check_evict(ctx, src, dst, lens, w, keep, 16, 500, None)


def test_eviction_updates_the_lengths_in_place(ctx):
    """The lengths' own array as the target: every head of a sequence has read its length by then."""
    B, H, cap, keep = 8, 16, 4096, 1000
    src, dst = tq.Cache(ctx, B, H, cap, device=DEV), tq.Cache(ctx, B, H, keep, device=DEV)
    lens = [4096, 3000, 1001, 1000, 999, 1, 0, 2222]
    fill(ctx, src, lens, 5)
    w = torch.rand(B, H, cap, generator=gen(1), device=DEV)
    want = [t.clone() for t in tq.tq_q8_evict(ctx.handle, src, dst, ints(lens), w, keep, 16, 500)]
    for _ in range(20):
        own = ints(lens)
        got = tq.tq_q8_evict(ctx.handle, src, dst, own, w, keep, 16, 500, dst_lens=own)
        assert got[1] is own and own.tolist() == [min(n, keep) for n in lens]
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_eviction_of_more_slots_than_shared_memory_holds(ctx):
    cap = 8 * 45056 + 30001  # the rest of each CTA's run is read again
    src, dst = tq.Cache(ctx, 1, 1, cap, device=DEV), tq.Cache(ctx, 1, 1, 200, device=DEV)
    w = torch.randn(1, 1, cap, generator=gen(8), device=DEV)
    kept, dlens, dw, dp = tq.tq_q8_evict(ctx.handle, src, dst, ints([cap - 3]), w, 200, 5, 20)
    np.testing.assert_array_equal(kept[0, 0].cpu().numpy(), q8.evict(w[0, 0].cpu().numpy(), cap - 3, 200, 5, 20))


def test_eviction_cuts_bad_lengths_and_reports_them(ctx):
    src, dst = paged(ctx, 2, 1, 128), tq.Cache(ctx, 2, 1, 64, device=DEV)
    fill(ctx, src, [128, 128], 5)
    w = torch.rand(2, 1, 128, generator=gen(1), device=DEV)
    check_evict(ctx, src, dst, [129, -4], w, 40, 1, 1, None)
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG


# ------------------------------------------------------------------------------------------------ refusals

def refused(status, f, *a, **kw):
    with pytest.raises(tq.TQError) as e:
        f(*a, **kw)
    assert e.value.status == status


def test_refusals(ctx):
    x = randn(1, 2, 3, 4, 128)
    pos = ints(np.zeros((2, 4)))
    refused(tq.TQ_ERR_STATE, tq.tq_rotary, ctx.handle, x, pos)
    for bad in (dict(dim=0), dict(dim=12), dict(dim=136), dict(base=1.0), dict(base=float("nan")), dict(factor=0.5), dict(gain=0.0),
                dict(factor=2.0, low=1.0, high=1.0), dict(factor=2.0, low=1.0, high=4.0)):
        refused(tq.TQ_ERR_ARG, tq.tq_set_rope, ctx.handle, **bad)
    cache = tq.Cache(ctx, 2, 3, 64, device=DEV)
    lens = ints([0, 0])
    refused(tq.TQ_ERR_STATE, tq.tq_q8_append, ctx.handle, cache, x, x, lens, rope=True)
    tq.tq_set_rope(ctx.handle)
    flat = torch.zeros(2 * 3 * 4 * 136, dtype=BF, device=DEV)
    odd = flat[:2 * 3 * 4 * 132].view(2, 3, 4, 132)[..., :128]  # rows 264 bytes apart
    refused(tq.TQ_ERR_ALIGN, tq.tq_rotary, ctx.handle, odd, pos)
    refused(tq.TQ_ERR_ALIGN, tq.tq_rotary, ctx.handle, flat[4:4 + x.numel()].view(x.shape), pos)
    refused(tq.TQ_ERR_ALIGN, tq.tq_q8_append, ctx.handle, cache, odd, odd, lens)
    refused(tq.TQ_ERR_ARG, tq.tq_rotary, ctx.handle, x, pos, out=x[:, :, :1].expand(2, 3, 4, 128))
    refused(tq.TQ_ERR_ARG, tq.tq_q8_append, ctx.handle, tq.Cache(ctx, 2, 4, 64, device=DEV), x, x, lens)
    with pytest.raises(ValueError):
        tq.tq_rotary(ctx.handle, x, pos.long())
    with pytest.raises(ValueError):
        tq.tq_rotary(ctx.handle, x.transpose(2, 3), pos)
    with pytest.raises(TypeError):
        tq.tq_rotary(ctx.handle, x.double(), pos)
    with pytest.raises(ValueError):
        tq.tq_q8_append(ctx.handle, cache, x, x.float(), lens)
    w = torch.zeros(2, 3, 64, device=DEV)
    dst = tq.Cache(ctx, 2, 3, 32, device=DEV)
    for keep, sink, recent in ((0, 0, 0), (33, 0, 0), (10, 6, 5), (10, -1, 0), (10, 0, -1)):
        refused(tq.TQ_ERR_ARG, tq.tq_q8_evict, ctx.handle, cache, dst, lens, w, keep, sink, recent)
    refused(tq.TQ_ERR_ARG, tq.tq_q8_evict, ctx.handle, cache, cache, lens, w, 10)
    other = tq.Context(128, 4, "KQV", 1)
    kqv = tq.Cache(other, 2, 3, 64, device=DEV)
    refused(tq.TQ_ERR_STATE, tq.tq_q8_append, other.handle, kqv, x, x, lens)
    for rotation in (tq.tq_set_rotation,):
        refused(tq.TQ_ERR_STATE, rotation, ctx.handle, "dense")
    refused(tq.TQ_ERR_ARG, tq.tq_init, 128, 4, "Q8", 1)
    other.close()
