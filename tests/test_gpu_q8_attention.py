"""Attention over the 8-bit cache on the GPU against fp64 attention over the values its codes stand
for (oracle/q8.py). The tolerance of every output is a bound on the kernels' roundings, computed per
element from the same inputs (see `check`)."""

import numpy as np
import pytest
import torch

from oracle import q8
from quantised_kv_cache_gb300 import tq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


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


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def np64(t):
    return t.double().cpu().numpy()


def make(ctx, B, H, cap, lens, seed=0, paged=False, poison=True, spread=0.5):
    """A cache of random tokens whose unwritten slots hold NaN codes, and the values it stands for."""
    if paged:
        n = B * H * (-(-cap // 64))
        table = torch.from_numpy(np.random.default_rng(seed).permutation(n + 5)[:n].astype(np.int32)).view(B, H, -1).to(DEV)
        cache = tq.PagedCache(ctx, B, H, cap, n + 5, table, device=DEV)
    else:
        cache = tq.Cache(ctx, B, H, cap, device=DEV)
    if poison:
        cache.tensors["records"].fill_(0x7f)
        for name in ("k_stats", "v_stats"):
            cache.tensors[name].view(F32).fill_(float("nan"))
    n = max(int(max(lens)), 1)
    k = torch.randn(B, H, n, 128, generator=gen(seed + 1), device=DEV) * torch.exp(spread * torch.randn(1, H, 1, 128, generator=gen(seed + 2), device=DEV))
    v = torch.randn(B, H, n, 128, generator=gen(seed + 3), device=DEV) * torch.exp(torch.randn(B, H, n, 1, generator=gen(seed + 4), device=DEV))
    tq.tq_q8_append(ctx.handle, cache, k.to(BF), v.to(BF), ints([0] * B), new_lens=ints(lens))
    kv, vv = tq.tq_dequantize(ctx.handle, cache, 0, cap)
    return cache, np64(kv), np64(vv)


def check(got, q, k, v, lens, new, *, dtype, out_dtype, begin=None, end=None, scale=None, softcap=0.0, slopes=None, q_pos=None,
          k_pos=None, lse=None, weights=None, before=None, rows=None):
    """Every element within the bound. Per query: the products' sums are off by at most 130 U of the sum of their magnitudes (fp32,
    any order, three scalings). A query enters as 8-bit terms with its row's largest coordinate in [128, 256): 16-bit
    coordinates of at least 2^-9 of the largest exactly, smaller ones within 2^-20 of it (for many rows three terms end at 2^-13, two, in
    bf16, at 2^-10: 2^-17; for few rows all terms are e5m2 and end far below), float32 ones within 2^-22 of themselves and 2^-31 of the largest (8 terms).
    Capping, bias and the exponent add a few U of what they handle (a cap by the short tanh of many rows 2^-21 of the cap); a probability's relative error is twice the
    largest score error (its own and the sum's) and 2^-20 for the two exponentials. Probabilities enter the value sums as terms of
    their 2^8-fold: 2^-11 of each and 2^-21 of the largest (three terms; four e5m2 ones do better), 2^-8 and 2^-18 (two, many rows in bf16), 2^-22 and 2^-32
    (8), never more than itself; many rows fold value scales up to 2^4 apart into them, which brings the second nearer by 2^4.
    Sums over tiles of 128 add U each; the result is rounded to its type."""
    B, Hq, n, _ = q.shape
    H = k.shape[1]
    G = Hq // H
    sc = 1 / np.sqrt(128.0) if scale is None else scale
    wide = out_dtype == F32
    many = G * n > 16 and not wide
    worst = 0.0
    wsum = np.zeros((B, H, k.shape[2])) if weights is not None else None
    wtol = np.zeros_like(wsum) if weights is not None else None
    for b in range(B):
        L, m = int(lens[b]), int(new[b])
        at = L - m + np.arange(m)
        lo = np.zeros(m, int) if begin is None else np.maximum(begin[b][:m], 0)
        hi = np.minimum(at + 1 if end is None else end[b][:m], L)
        for hq in range(Hq):
            if rows is not None and (b, hq) not in rows:
                continue
            h = hq // G
            qq, kk, vv = q[b, hq, :m], np.nan_to_num(k[b, h, :L]), np.nan_to_num(v[b, h, :L])
            qp = at if q_pos is None else q_pos[b][:m]
            kp = np.arange(L) if k_pos is None else k_pos[b, h, :L]
            sl = 0.0 if slopes is None else float(slopes[hq])
            want, p, wl = q8.attend(qq, kk, vv, lo, hi, scale=sc, softcap=softcap, slope=sl, q_pos=qp, k_pos=kp)
            if L == 0 or m == 0:
                assert not got[b, hq, :m].any()
                continue
            big = np.abs(qq).max(-1, keepdims=True)
            if dtype == F32:
                dq = 2.0 ** -22 * np.abs(qq) + 2.0 ** -31 * big
            else:
                dq = np.where(np.abs(qq) < 2.0 ** -9 * big, (2.0 ** -31 if wide else 2.0 ** -17 if many and dtype == BF else 2.0 ** -20) * big, 0.0)
            e = sc * (dq @ np.abs(kk).T) + 130 * U * sc * (np.abs(qq) @ np.abs(kk).T)
            dist = np.abs(qp[:, None] - kp[None])
            e = e + 8 * U * (softcap * (2 if many else 1) + np.abs(sl * dist) + sc * np.abs(qq @ kk.T))
            e = np.where(p > 0, e, 0).max(-1, keepdims=True) if L else e
            rel = 2 * e + 2.0 ** -20
            term, floor = (2.0 ** -22, 2.0 ** -32) if wide else (2.0 ** -8, 2.0 ** -14) if many and dtype == BF else (2.0 ** -11, 2.0 ** -17 if many else 2.0 ** -21)
            mass = p @ np.abs(vv)
            tol = (rel + 2 * (140 + L / 128) * U) * mass
            tol += 2 * (np.minimum(p, term * p + floor * p.max(-1, keepdims=True)) @ np.abs(vv)) + np.abs(want) * torch.finfo(out_dtype).eps / 2 * 1.01
            tol += 1e-30 if wide or out_dtype == BF else 2.0 ** -25
            err = np.abs(got[b, hq, :m] - want)
            # a number from half a step past the type's largest on rounds to infinity
            past = np.abs(want) + tol >= float(torch.finfo(out_dtype).max) * (1 + torch.finfo(out_dtype).eps / 4)
            err = np.where(past & (got[b, hq, :m] == np.where(want < 0, -np.inf, np.inf)), 0.0, err)
            assert np.all(err <= tol), (b, hq, (err / tol).max())
            worst = max(worst, (err / tol).max())
            if lse is not None:
                empty = np.isneginf(wl)
                assert np.array_equal(np.isneginf(lse[b, hq, :m]), empty)
                d = np.abs(lse[b, hq, :m][~empty] - wl[~empty])
                assert np.all(d <= (e[:, 0] + 2.0 ** -20 + (140 + L / 128) * U + 4 * U * np.abs(wl))[~empty])
            if weights is not None:
                wsum[b, h, :L] += p.sum(0)
                wtol[b, h, :L] += (p * (rel + 2.0 ** -19 + 4 * (140 + L / 128) * U)).sum(0) + 2.0 ** -126
    if weights is not None:
        base = np.zeros_like(wsum) if before is None else before
        assert np.all(np.abs(weights - base - wsum) <= wtol + (G * n + 2) * U * (np.abs(base) + wsum))
    return worst


def queries(seed, B, Hq, n, dtype, layout="heads", size=1.0):
    x = torch.randn(B, Hq, n, 128, generator=gen(seed), device=DEV) * size
    if layout == "tokens":
        return x.transpose(1, 2).contiguous().to(dtype).transpose(1, 2)
    return x.to(dtype)


CASES = [  # B, heads_q, heads_kv, n_q, lens
    (1, 1, 1, 1, [1]), (1, 1, 1, 1, [2]), (2, 4, 4, 1, [31, 64]), (1, 8, 8, 1, [33]), (3, 8, 2, 1, [65, 127, 128]),
    (2, 12, 4, 1, [129, 500]), (4, 14, 2, 1, [1, 192, 0, 700]), (1, 32, 4, 1, [1000]), (2, 32, 2, 1, [513, 90]),
    (2, 40, 2, 1, [300, 77]), (1, 6, 2, 2, [200]), (2, 4, 4, 5, [5, 130]), (2, 8, 4, 7, [64, 300]), (1, 16, 2, 4, [257]),
    (1, 8, 2, 33, [300]), (40, 2, 2, 1, [1 + 13 * i for i in range(40)]), (1, 1, 1, 1, [30000]), (1, 4, 1, 1, [20001]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:4])) + f"-{max(c[4])}")
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, HF), (F32, F32), (BF, F32), (HF, F32)])
def test_causal_attention(ctx, case, dtype, out):
    B, Hq, H, n, lens = case
    cap = max(max(lens), n) + 70
    cache, k, v = make(ctx, B, H, cap, lens, seed=sum(lens), paged=sum(lens) % 2 == 1)
    q = queries(5, B, Hq, n, dtype, "tokens" if B % 2 else "heads")
    lse = torch.empty(B, Hq, n, device=DEV)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, lse=lse, out_dtype=out)
    assert got.dtype == out
    check(np64(got), np64(q), k, v, lens, [n] * B, dtype=dtype, out_dtype=out, lse=np64(lse))


PROMPTS = [  # B, heads_q, heads_kv, n_q, lens
    (1, 1, 1, 65, [65]), (1, 1, 1, 128, [128]), (2, 2, 1, 129, [129, 1]), (1, 4, 1, 64, [64]), (1, 8, 2, 200, [1000]),
    (3, 3, 1, 100, [100, 300, 163]), (2, 14, 2, 77, [400, 77]), (1, 16, 1, 257, [300]), (5, 4, 4, 70, [70, 71, 700, 128, 191]),
    (1, 2, 2, 1000, [1300]), (1, 1, 1, 70, [9000]),
]


@pytest.mark.parametrize("case", [(4, 16, 8, 10, [700, 0, 1, 129], 7500), (4, 8, 8, 128, [300, 128, 1000, 131], 7500), (2, 64, 8, 8, [900, 65], 14720),
                                  (1, 40, 8, 5, [29000], 30000), (30, 18, 1, 1, [64 * i for i in range(30)], 8000)],
                         ids=lambda c: "-".join(map(str, c[:4])) + f"-{max(c[4])}")
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("extra", ["plain", "masked capped biased paged"])
def test_rows_of_one_tile_over_many_slots(ctx, case, dtype, extra):
    """Enough slots for two units a CTA at once, each with half of the ring: mostly beyond the sequences, or really long."""
    B, Hq, H, n, lens, cap = case
    assert 16 < Hq // H * n <= 128 and B * H * -(-cap // 128) >= 12 * torch.cuda.get_device_properties(0).multi_processor_count
    cache, k, v = make(ctx, B, H, cap, lens, seed=sum(lens), paged=extra != "plain", poison=False)
    q = queries(5, B, Hq, n, dtype, "tokens")
    kw, ck, new = {}, {}, [min(n, L) for L in lens]
    if extra != "plain":
        rng = np.random.default_rng(n)
        ck = dict(begin=rng.integers(-5, 100, (B, n)), end=rng.integers(0, 2 * max(lens), (B, n)), softcap=15.0)
        slopes = torch.linspace(0.01, 0.2, Hq, device=DEV)
        kw = dict(key_begin=ints(ck["begin"]), key_end=ints(ck["end"]), softcap=15.0, slopes=slopes)
        ck["slopes"] = slopes.double().cpu().numpy()
    lse, out = torch.zeros(B, Hq, n, device=DEV), torch.full_like(q, 77.0)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, new_lens=ints(new), lse=lse, out=out, **kw)
    check(np64(got), np64(q), k, v, lens, new, dtype=dtype, out_dtype=dtype, lse=np64(lse), **ck)
    for b in range(B):
        assert bool((got[b, :, new[b]:] == 77).all())


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: "-".join(map(str, c[:4])) + f"-{max(c[4])}")
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, HF), (F32, F32)])
def test_prompts(ctx, case, dtype, out):
    B, Hq, H, n, lens = case
    cap = max(max(lens), n) + 70
    cache, k, v = make(ctx, B, H, cap, lens, seed=sum(lens), paged=sum(lens) % 2 == 1)
    q = queries(5, B, Hq, n, dtype, "tokens" if B % 2 else "heads")
    lse = torch.empty(B, Hq, n, device=DEV)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, lse=lse, out_dtype=out)
    check(np64(got), np64(q), k, v, lens, [n] * B, dtype=dtype, out_dtype=out, lse=np64(lse))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompts_whose_blocks_have_far_apart_values(ctx, dtype):
    """Value scales of neighbouring blocks differ by up to 2^16, a block of zeros among them."""
    B, Hq, H, n, N, cap = 1, 6, 2, 90, 640, 704
    cache = tq.Cache(ctx, B, H, cap, device=DEV)
    k, v = queries(1, B, H, N, BF), torch.randn(B, H, N, 128, generator=gen(2), device=DEV)
    for j, e in enumerate([0, 16, 12, 8, 3, 0, 0, -8, 5, 5]):
        v[:, :, 64 * j:64 * j + 64] *= 2.0 ** e if j != 6 else 0.0
    tq.tq_q8_append(ctx.handle, cache, k, v.to(BF), ints([0]))
    kv, vv = (np64(t) for t in tq.tq_dequantize(ctx.handle, cache, 0, cap))
    q = queries(3, B, Hq, n, dtype)
    rng = np.random.default_rng(1)
    begin = rng.integers(0, N, (B, n))
    end = np.minimum(begin + rng.integers(1, 200, (B, n)), N)
    for kw in ({}, dict(key_begin=ints(begin), key_end=ints(end))):
        got = tq.tq_q8_attention(ctx.handle, cache, q, ints([N]), cap, out_dtype=dtype, **kw)
        check(np64(got), np64(q), kv, vv, [N], [n], dtype=dtype, out_dtype=dtype, begin=begin if kw else None, end=end if kw else None)


def test_prompts_over_unmapped_blocks():
    ctx = tq.Context(128, 8, "Q8", 1)
    cache, k, v = make(ctx, 1, 2, 320, [300], seed=4, paged=True)
    q = queries(5, 1, 4, 80, BF)
    cache.block_table[0, 0, 1], cache.block_table[0, 1, 4] = -1, cache.pool_blocks
    cache.block_table[0, 1, 2], cache.block_table[0, 1, 3] = -1, -1
    end = ints([[300] * 80])
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([300]), 320, key_end=end)
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    k2, v2 = np.concatenate([k[:, :1, :64], k[:, :1, 128:300]], 2), np.concatenate([v[:, :1, :64], v[:, :1, 128:300]], 2)
    check(np64(got[:, :2]), np64(q[:, :2]), k2, v2, [236], [80], dtype=BF, out_dtype=BF, end=[[236] * 80])
    check(np64(got[:, 2:]), np64(q[:, 2:]), k[:, 1:], v[:, 1:], [128], [80], dtype=BF, out_dtype=BF, end=[[128] * 80])
    ctx.close()


@pytest.mark.parametrize("softcap,bias,mask,positions", [
    (20.0, False, "causal", False), (0.0, True, "causal", False), (30.0, True, "window", False), (0.0, False, "window", False),
    (0.0, False, "documents", False), (5.0, True, "documents", True), (0.0, True, "causal", True), (0.0, False, "empty", False)])
@pytest.mark.parametrize("B,Hq,H,n,lens,new", [(2, 4, 2, 1, [400, 3], None), (3, 8, 2, 6, [300, 6, 0], [6, 4, 0]), (2, 6, 2, 40, [333, 129], [40, 17])])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_caps_biases_and_masks(ctx, softcap, bias, mask, positions, B, Hq, H, n, lens, new, dtype):
    cap = 448
    rng = np.random.default_rng(n)
    cache, k, v = make(ctx, B, H, cap, lens, seed=7)
    q = queries(6, B, Hq, n, dtype, "tokens", size=3.0)
    m = [n] * B if new is None else new
    begin = end = None
    if mask == "window":
        at = np.array([np.arange(n) + L - w for L, w in zip(lens, m)])
        begin, end = at - rng.integers(0, 200, at.shape), at + 1
    elif mask == "documents":  # any range: before the start, past the end, reversed
        begin, end = rng.integers(-5, 300, (B, n)), rng.integers(0, 500, (B, n))
    elif mask == "empty":
        begin, end = rng.integers(100, 200, (B, n)), rng.integers(0, 101, (B, n))
    kw = {}
    if bias:
        kw["slopes"] = torch.linspace(0.5, 0.001, Hq, device=DEV)
    if positions:
        kw["q_positions"] = ints(rng.integers(-2 ** 20, 2 ** 20, (B, n)))
        kw["k_positions"] = ints(rng.integers(-2 ** 20, 2 ** 20, (B, H, cap)))
        kw["slopes"] = kw["slopes"] * 2.0 ** -20
    out = torch.full(q.shape, 77.0, device=DEV, dtype=dtype)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, new_lens=None if new is None else ints(new), softcap=softcap,
                             scale=0.05, key_begin=None if begin is None else ints(begin), key_end=None if end is None else ints(end), out=out, **kw)
    check(np64(got), np64(q), k, v, lens, m, dtype=dtype, out_dtype=dtype, begin=begin, end=end, scale=0.05, softcap=softcap,
          slopes=None if not bias else kw["slopes"].cpu().numpy(), q_pos=None if not positions else kw["q_positions"].cpu().numpy(),
          k_pos=None if not positions else kw["k_positions"].cpu().numpy())
    for b in range(B):  # rows behind a sequence's query tokens
        assert bool((got[b, :, m[b]:] == 77).all())


@pytest.mark.parametrize("case", [(1, 1, 1, 1, [1]), (3, 8, 2, 1, [65, 0, 128]), (2, 40, 2, 1, [300, 77]), (2, 4, 4, 5, [5, 130]),
                                  (1, 8, 2, 33, [300]), (2, 16, 4, 100, [260, 100]), (1, 32, 8, 1, [1000]), (16, 4, 4, 1, [50 * i + 1 for i in range(16)])],
                         ids=lambda c: "-".join(map(str, c[:4])) + f"-{max(c[4])}")
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("extra", ["plain", "ragged masked capped biased paged"])
def test_accumulated_weights(ctx, case, dtype, extra):
    B, Hq, H, n, lens = case
    cap = max(max(lens), n) + 70
    cache, k, v = make(ctx, B, H, cap, lens, seed=sum(lens), paged=extra != "plain")
    q = queries(5, B, Hq, n, dtype, "tokens")
    new, kw, ck = [n] * B, {}, {}
    if extra != "plain":
        rng = np.random.default_rng(n)
        new = [int(rng.integers(0, n + 1)) for _ in range(B)]
        ck = dict(begin=rng.integers(-5, 100, (B, n)), end=rng.integers(0, 400, (B, n)), softcap=15.0, slopes=np.linspace(0.01, 0.3, Hq))
        kw = dict(key_begin=ints(ck["begin"]), key_end=ints(ck["end"]), softcap=15.0, slopes=torch.as_tensor(ck["slopes"], dtype=F32, device=DEV),
                  new_lens=ints(new))
        ck["slopes"] = kw["slopes"].double().cpu().numpy()
    before = torch.rand(B, H, cap, generator=gen(8), device=DEV)
    out = torch.zeros_like(q)
    alone = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, out=out, **kw).clone()
    both = torch.full_like(before, float("nan"))
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, weights_in=before, weights=both, out=out, **kw)
    assert torch.equal(got, alone)
    check(np64(got), np64(q), k, v, lens, new, dtype=dtype, out_dtype=dtype, weights=np64(both), before=np64(before), **ck)
    fresh = torch.full_like(before, float("nan"))
    tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, weights=fresh, out=out, **kw)
    check(np64(got), np64(q), k, v, lens, new, dtype=dtype, out_dtype=dtype, weights=np64(fresh), **ck)
    place = before.clone()
    tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, weights_in=place, weights=place, out=out, **kw)
    assert torch.equal(place, both)


def test_a_served_sequence_from_prompt_to_eviction_and_on(ctx):
    """A prompt is appended and attended, a few tokens are decoded while their attention weight accumulates, the cache is cut by it,
    and decoding goes on over the kept tokens at their old positions."""
    B, Hq, H, n, cap, keep = 2, 8, 2, 200, 320, 128
    tq.tq_set_rope(ctx.handle, 64, interleaved=True)
    cache, dst = tq.Cache(ctx, B, H, cap, device=DEV), tq.Cache(ctx, B, H, 192, device=DEV)
    model = {"k": q8.Model(B * H, cap), "v": q8.Model(B * H, cap)}
    lens = np.zeros(B, int)
    w = torch.zeros(B, H, cap, device=DEV)
    slopes = torch.tensor([2.0 ** -(i + 1) for i in range(Hq)], device=DEV)

    def tokens(seed, m):
        return [queries(seed + i, B, x, m, BF, "tokens") for i, x in enumerate((Hq, H, H))]

    for step, m in enumerate([n] + [1] * 5):
        q, k, v = tokens(100 * step, m)
        pos = ints(lens[:, None] + np.arange(m))
        qr = tq.tq_rotary(ctx.handle, q, pos)
        kr = tq.tq_rotary(ctx.handle, k, pos)
        tq.tq_q8_append(ctx.handle, cache, k, v, ints(lens), rope=True)
        for b in range(B):
            for h in range(H):
                model["k"].append(b * H + h, int(lens[b]), np64(kr)[b, h])
                model["v"].append(b * H + h, int(lens[b]), np64(v)[b, h])
        lens = lens + m
        before = np64(w)
        out = tq.tq_q8_attention(ctx.handle, cache, qr, ints(lens), cap, slopes=slopes, weights_in=w, weights=w)
        kv, vv = (x.values().reshape(B, H, -1, 128)[:, :, :cap] for x in (model["k"], model["v"]))
        check(np64(out), np64(qr), kv, vv, lens, [m] * B, dtype=BF, out_dtype=BF, slopes=np64(slopes), weights=np64(w), before=before)
    kept, dlens, dw, dp = tq.tq_q8_evict(ctx.handle, cache, dst, ints(lens), w, keep, 4, 16)
    wn = w.cpu().numpy()
    km, vm = q8.Model(B * H, 192), q8.Model(B * H, 192)
    places = np.zeros((B, H, 192), int)
    for b in range(B):
        for h in range(H):
            stay = q8.evict(wn[b, h], int(lens[b]), keep, 4, 16)
            np.testing.assert_array_equal(kept[b, h].cpu().numpy(), stay)
            places[b, h, :keep] = stay
            km.append(b * H + h, 0, kv[b, h, stay])
            vm.append(b * H + h, 0, vv[b, h, stay])
    q, k, v = tokens(9000, 1)
    pos = ints(lens[:, None])
    qr, kr = tq.tq_rotary(ctx.handle, q, pos), tq.tq_rotary(ctx.handle, k, pos)
    tq.tq_q8_append(ctx.handle, dst, k, v, dlens, rope=True, positions=pos)
    dp[torch.arange(B)[:, None], torch.arange(H)[None], dlens.long()[:, None]] = pos.expand(B, H)
    for b in range(B):
        for h in range(H):
            km.append(b * H + h, keep, np64(kr)[b, h])
            vm.append(b * H + h, keep, np64(v)[b, h])
            places[b, h, keep] = lens[b]
    out = tq.tq_q8_attention(ctx.handle, dst, qr, dlens + 1, 192, slopes=slopes, q_positions=pos, k_positions=dp, weights_in=dw, weights=dw)
    check(np64(out), np64(qr), km.values().reshape(B, H, -1, 128), vm.values().reshape(B, H, -1, 128), [keep + 1] * B, [1] * B, dtype=BF,
          out_dtype=BF, slopes=np64(slopes), q_pos=lens[:, None], k_pos=places)


def test_layouts_and_paging_give_the_same_bits(ctx):
    B, Hq, H, n, lens = 3, 8, 4, 2, [500, 130, 64]
    plain, _, _ = make(ctx, B, H, 512, lens, seed=3)
    pages, _, _ = make(ctx, B, H, 512, lens, seed=3, paged=True)
    q = queries(5, B, Hq, n, BF)
    want = tq.tq_q8_attention(ctx.handle, plain, q, ints(lens), 512)
    assert torch.equal(tq.tq_q8_attention(ctx.handle, pages, q, ints(lens), 512), want)
    wide = torch.full((n, Hq, B, 160), 5.0, dtype=BF, device=DEV)
    view = wide[..., 16:144].permute(2, 1, 0, 3)
    view.copy_(q)
    out = torch.full((B, n, Hq, 136), 9.0, dtype=BF, device=DEV)
    tq.tq_q8_attention(ctx.handle, pages, view, ints(lens), 512, out=out[..., :128].transpose(1, 2))
    assert torch.equal(out[..., :128].transpose(1, 2), want) and bool((out[..., 128:] == 9).all())
    one = tq.tq_q8_attention(ctx.handle, plain, q[:, :, :1].expand(B, Hq, 1, 128), ints(lens), 512)
    assert one.shape == (B, Hq, 1, 128)


def test_the_general_calls_take_the_8_bit_cache(ctx):
    """tq_decode_attention and tq_decode_step equal the append and the attention call they stand for."""
    B, Hq, H, cap, lens = 3, 8, 2, 320, [255, 64, 0]
    a, k, v = make(ctx, B, H, cap, lens, seed=9, poison=False)
    b, _, _ = make(ctx, B, H, cap, lens, seed=9, poison=False)
    q = queries(5, B, Hq, 1, BF)
    kn, vn = queries(6, B, H, 1, BF, size=4.0), queries(7, B, H, 1, BF, size=4.0)
    got = tq.tq_decode_attention(ctx.handle, a, q[:, :, 0].contiguous(), ints(lens), cap)
    want = tq.tq_q8_attention(ctx.handle, a, q, ints(lens), cap, key_end=ints([[n] for n in lens]), out_dtype=F32)
    assert torch.equal(got, want[:, :, 0])
    check(np64(want), np64(q), k, v, lens, [1] * B, dtype=BF, out_dtype=F32, end=[[n] for n in lens])
    step = tq.tq_decode_step(ctx.handle, a, q[:, :, 0].contiguous(), kn, vn, ints(lens), cap)
    tq.tq_q8_append(ctx.handle, b, kn, vn, ints(lens))
    more = ints([n + 1 for n in lens])
    assert torch.equal(step, tq.tq_q8_attention(ctx.handle, b, q, more, cap, out_dtype=F32)[:, :, 0])
    for name in a.tensors:
        assert torch.equal(a.tensors[name], b.tensors[name])
    static = tq.tq_decode_attention_static(ctx.handle, a, q[:, :, 0].contiguous(), more, cap)
    assert torch.equal(static, step)


def test_queries_that_are_not_finite_spoil_their_own_rows_only(ctx):
    cache, k, v = make(ctx, 1, 2, 256, [200], seed=2)
    q = queries(5, 1, 8, 3, BF)
    want = tq.tq_q8_attention(ctx.handle, cache, q, ints([200]), 256)
    q[0, 1, 1, 5], q[0, 6, 2, 0] = float("nan"), float("inf")
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([200]), 256)
    bad = torch.zeros(1, 8, 3, 128, dtype=torch.bool, device=DEV)
    bad[0, 1, 1] = bad[0, 6, 2] = True
    assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], want[~bad])


def test_large_scores_small_scores_and_far_maxima(ctx):
    """Rows whose maximum comes in the first, a middle or the last tile, scores of +-1000, all-equal scores."""
    cap, H = 1536, 1
    k = torch.zeros(1, 1, cap, 128, device=DEV)
    v = torch.randn(1, 1, cap, 128, generator=gen(1), device=DEV)
    k[0, 0, :, 0] = 0.01 * torch.randn(cap, generator=gen(2), device=DEV)
    for i, at in enumerate((0, 127, 128, 700, cap - 1)):
        k[0, 0, at, 1 + i] = 100.0
    cache = tq.Cache(ctx, 1, H, cap, device=DEV)
    tq.tq_q8_append(ctx.handle, cache, k.to(BF), v.to(BF), ints([0]))
    kv, vv = (np64(t) for t in tq.tq_dequantize(ctx.handle, cache, 0, cap))
    q = torch.zeros(1, 8, 1, 128, device=DEV)
    for i in range(5):
        q[0, i, 0, 1 + i] = 100.0 if i % 2 else -100.0
    q[0, 5, 0, 0] = 1e-30
    q[0, 6, 0, 0] = 50.0
    for dt in (BF, F32):
        got = tq.tq_q8_attention(ctx.handle, cache, q.to(dt), ints([cap]), cap)
        check(np64(got), np64(q.to(dt)), kv, vv, [cap], [1], dtype=dt, out_dtype=dt)


def test_a_block_table_that_lies_is_reported_and_its_tokens_are_unseen():
    ctx = tq.Context(128, 8, "Q8", 1)
    cache, k, v = make(ctx, 1, 2, 320, [300], seed=4, paged=True)
    q = queries(5, 1, 4, 1, BF)
    cache.block_table[0, 0, 1], cache.block_table[0, 1, 4] = -1, cache.pool_blocks
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([300]), 320)
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    k2, v2 = np.concatenate([k[:, :1, :64], k[:, :1, 128:300]], 2), np.concatenate([v[:, :1, :64], v[:, :1, 128:300]], 2)
    check(np64(got[:, :2]), np64(q[:, :2]), k2, v2, [236], [1], dtype=BF, out_dtype=BF)
    check(np64(got[:, 2:]), np64(q[:, 2:]), k[:, 1:], v[:, 1:], [256], [1], dtype=BF, out_dtype=BF)
    # lengths outside their range are cut
    tq.tq_q8_attention(ctx.handle, cache, q, ints([321]), 320)
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    tq.tq_q8_attention(ctx.handle, cache, q, ints([-1]), 320)
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    tq.tq_q8_attention(ctx.handle, cache, q, ints([64]), 320, new_lens=ints([2]))
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    ctx.close()


def test_guards_around_the_output_and_the_workspace(ctx):
    B, Hq, H, n, lens = 2, 8, 2, 3, [700, 90]
    cache, _, _ = make(ctx, B, H, 704, lens, seed=4)
    q = queries(5, B, Hq, n, BF)
    need = tq.tq_q8_attention_workspace(ctx.handle, B, Hq, H, n, 704)
    ws = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((B * Hq * n * 128 + 256,), 3.0, dtype=BF, device=DEV)
    want = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), 704)
    tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), 704, workspace=ws[4096:4096 + need], out=out[128:-128].view(q.shape))
    assert torch.equal(out[128:-128].view(q.shape), want)
    assert bool((ws[:4096] == 0xA5).all()) and bool((ws[4096 + need:] == 0xA5).all())
    assert bool((out[:128] == 3).all()) and bool((out[-128:] == 3).all())


def test_two_streams_and_replayed_graphs(ctx):
    """Two attention calls at once on streams of their own, and a captured rotary-append-attend step replayed with changed inputs."""
    B, Hq, H, cap, lens = 4, 16, 4, 1024, [1000, 3, 500, 64]
    tq.tq_set_rope(ctx.handle)
    caches = [make(ctx, B, H, cap, lens, seed=s, poison=False)[0] for s in (1, 2)]
    q = [queries(s, B, Hq, 1, BF) for s in (3, 4)]
    want = [tq.tq_q8_attention(ctx.handle, c, x, ints(lens), cap) for c, x in zip(caches, q)]
    L = ints(lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for s, c, x in zip(streams, caches, q):
            with torch.cuda.stream(s):
                got.append(tq.tq_q8_attention(ctx.handle, c, x, L, cap))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the step as a graph
    k, v = queries(8, B, H, 1, BF), queries(9, B, H, 1, BF)
    pos, now, later = L[:, None].contiguous(), L.clone(), L + 1
    ws = torch.empty(tq.tq_q8_attention_workspace(ctx.handle, B, Hq, H, 1, cap), dtype=torch.uint8, device=DEV)
    qr, out = torch.empty_like(q[0]), torch.empty_like(q[0])

    def step(cache):
        tq.tq_rotary(ctx.handle, q[0], pos, out=qr)
        tq.tq_q8_append(ctx.handle, cache, k, v, now, rope=True)
        tq.tq_q8_attention(ctx.handle, cache, qr, later, cap, workspace=ws, out=out)

    twin = make(ctx, B, H, cap, lens, seed=1, poison=False)[0]
    g = torch.cuda.CUDAGraph()
    step(twin)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(caches[0])
    for i in range(3):
        q[0].copy_(queries(20 + i, B, Hq, 1, BF))
        k.copy_(queries(30 + i, B, H, 1, BF))
        g.replay()
        got = out.clone()
        step(twin)
        assert torch.equal(got, out)
        now += 1
        later += 1
        pos += 1
    for name in twin.tensors:
        assert torch.equal(twin.tensors[name], caches[0].tensors[name])


@pytest.mark.parametrize("B,Hq,H,n,lens,dtype", [
    (600, 2, 1, 1, [1 + (37 * i) % 200 for i in range(600)], BF),   # more sequences than one launch takes
    (3, 2, 1, 2100, [2100, 2101, 2200], F32)])                      # more row tiles than one launch takes
def test_more_units_than_one_launch_takes(ctx, B, Hq, H, n, lens, dtype):
    cap = max(lens)
    cache, k, v = make(ctx, B, H, cap, lens, seed=1)
    q = queries(5, B, Hq, n, dtype)
    w = torch.zeros(B, H, cap, device=DEV)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, weights=w)
    if n > 1:  # the last rows
        m = 40
        check(np64(got[:, :, -m:]), np64(q[:, :, -m:]), k, v, lens, [m] * B, dtype=dtype, out_dtype=dtype)
        assert abs(float(w.sum()) / (B * Hq * n) - 1) < 1e-4
    else:
        check(np64(got), np64(q), k, v, lens, [1] * B, dtype=dtype, out_dtype=dtype, weights=np64(w))


def test_no_query_tokens_at_all(ctx):
    cache, _, _ = make(ctx, 2, 2, 128, [100, 5], seed=1)
    for n in (1, 3, 100):
        q = queries(5, 2, 4, n, BF)
        out, w = torch.full_like(q, 5.0), torch.ones(2, 2, 128, device=DEV)
        tq.tq_q8_attention(ctx.handle, cache, q, ints([100, 5]), 128, new_lens=ints([0, 0]), out=out, weights_in=w, weights=w)
        assert bool((out == 5).all()) and bool((w == 1).all())


def test_weights_of_more_scores_than_are_kept(ctx):
    """64 rows over a million slots: the scores are formed again."""
    N, cap, m = 1_049_000, 1_050_000, 200
    cache = tq.Cache(ctx, 1, 1, cap, device=DEV)
    k, v = queries(1, 1, 1, m, BF), queries(2, 1, 1, m, BF)
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([N - m]))
    q = queries(3, 1, 16, 4, BF)
    begin, end = ints([[N - m] * 4]), ints([[N - 3 + i for i in range(4)]])
    w = torch.zeros(1, 1, cap, device=DEV)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([N]), cap, key_begin=begin, key_end=end, weights=w)
    kv, vv = (np64(t) for t in tq.tq_dequantize(ctx.handle, cache, N - m, N))
    check(np64(got), np64(q), kv, vv, [m], [4], dtype=BF, out_dtype=BF, weights=np64(w[..., N - m:N]))
    assert not bool(w[..., :N - m].any()) and not bool(w[..., N:].any())


@pytest.mark.parametrize("case", [(1, 4, 1, 700, [900]), (1, 8, 1, 1100, [1300]), (2, 4, 2, 130, [257, 200]), (1, 8, 8, 40, [513]), (3, 20, 2, 2, [256, 1, 0]),
                                  (16, 8, 4, 70, [500 + 9 * i for i in range(16)])], ids=lambda c: "-".join(map(str, c[:4])) + f"-{max(c[4])}")
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("extra", ["causal", "documents", "capped biased", "placed"])
def test_weights_of_many_rows(ctx, case, dtype, extra):
    """Row tiles that are split over CTAs, that fill the ring many times, that see none of a CTA's tokens, that end early."""
    B, Hq, H, n, lens = case
    cap = max(lens) + 90
    cache, k, v = make(ctx, B, H, cap, lens, seed=sum(lens), paged=extra == "placed")
    q = queries(5, B, Hq, n, dtype, "tokens")
    kw, ck, new = {}, {}, [min(n, L) for L in lens]
    at = np.array([[L - m + i for i in range(n)] for L, m in zip(lens, new)])
    if extra == "documents":
        ck = dict(begin=np.maximum(at // 190 * 190, 0), end=at + 1)
        kw = dict(key_begin=ints(ck["begin"]), key_end=ints(ck["end"]))
    elif extra != "causal":
        slopes = torch.linspace(0.01, 0.2, Hq, device=DEV)
        ck, kw = dict(softcap=15.0, slopes=slopes.double().cpu().numpy()), dict(softcap=15.0, slopes=slopes)
        if extra == "placed":
            rng = np.random.default_rng(n)
            ck.update(q_pos=rng.integers(0, 500, (B, n)), k_pos=rng.integers(0, 500, (B, H, cap)))
            kw.update(q_positions=ints(ck["q_pos"]), k_positions=ints(ck["k_pos"]))
    before = torch.rand(B, H, cap, generator=gen(8), device=DEV)
    w, out = torch.full_like(before, float("nan")), torch.zeros_like(q)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, new_lens=ints(new), weights_in=before, weights=w, out=out, **kw)
    check(np64(got), np64(q), k, v, lens, new, dtype=dtype, out_dtype=dtype, weights=np64(w), before=np64(before), **ck)
    for b, L in enumerate(lens):
        assert torch.equal(w[b, :, L:], before[b, :, L:])
    place = before.clone()
    tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, new_lens=ints(new), weights_in=place, weights=place, out=out, **kw)
    assert torch.equal(place, w)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_weights_of_few_rows_and_more_slots_than_scores_are_kept_for(ctx, dtype):
    """128 heads over two million slots, nearly all beyond the sequence: more than a GB of scores would be kept."""
    H, cap, n = 8, 2_100_000, 300
    nblk = -(-cap // 64)
    table = torch.zeros(1, H, nblk, dtype=torch.int32, device=DEV)
    table[0, :, :8] = torch.arange(8 * H, device=DEV, dtype=torch.int32).flip(0).view(H, 8)
    cache = tq.PagedCache(ctx, 1, H, cap, pool_blocks=8 * H, block_table=table)
    k, v = queries(1, 1, H, n, BF), queries(2, 1, H, n, BF)
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([0]))
    q = queries(3, 1, 128, 1, dtype)
    assert 128 * cap * 4 > 1 << 30
    w = torch.zeros(1, H, cap, device=DEV)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([n]), cap, weights_in=w, weights=w)
    kv, vv = (np64(t) for t in tq.tq_dequantize(ctx.handle, cache, 0, n))
    check(np64(got), np64(q), kv, vv, [n], [1], dtype=dtype, out_dtype=dtype, weights=np64(w[..., :n]))
    assert not bool(w[..., n:].any())


@pytest.mark.parametrize("B,Hq,H,n,N", [(1, 8, 1, 300, 1000), (4, 32, 8, 8, 3000), (16, 16, 16, 20, 700)])
def test_back_to_back_weights_give_the_same_bits(ctx, B, Hq, H, n, N):
    cache = tq.Cache(ctx, B, H, N, device=DEV)
    k = queries(1, B, H, N, BF)
    tq.tq_q8_append(ctx.handle, cache, k, k, ints([0] * B))
    lens = ints([N] * B)
    for dtype in (BF, HF):
        q = queries(2, B, Hq, n, dtype)
        ws = torch.empty(tq.tq_q8_attention_workspace(ctx.handle, B, Hq, H, n, N, weights=True), dtype=torch.uint8, device=DEV)
        out, want = torch.empty_like(q), torch.empty(B, H, N, device=DEV)
        tq.tq_q8_attention(ctx.handle, cache, q, lens, N, workspace=ws, out=out, weights=want)
        w, bad = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device=DEV)
        for i in range(300):
            tq.tq_q8_attention(ctx.handle, cache, q, lens, N, workspace=ws, out=out, weights=w)
            if i % 25 == 24:
                bad += (w != want).sum()
        assert int(bad) == 0


@pytest.mark.parametrize("B,Hq,H,n,N", [(8, 32, 32, 1, 4096), (2, 32, 8, 1, 20000), (1, 16, 8, 300, 5000), (8, 32, 8, 8, 4000)])
def test_back_to_back_calls_give_the_same_bits(ctx, B, Hq, H, n, N):
    """Many calls without a pause between them: tiles' copies land in any order, CTAs follow one another on an SM."""
    cache = tq.Cache(ctx, B, H, N, device=DEV)
    k = queries(1, B, H, N, BF)
    tq.tq_q8_append(ctx.handle, cache, k, k, ints([0] * B))
    lens = ints([N] * B)
    for dtype in (BF, F32) if n == 1 else (BF, HF):
        q = queries(2, B, Hq, n, dtype)
        ws = torch.empty(tq.tq_q8_attention_workspace(ctx.handle, B, Hq, H, n, N), dtype=torch.uint8, device=DEV)
        want = tq.tq_q8_attention(ctx.handle, cache, q, lens, N, workspace=ws).clone()
        out, bad = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device=DEV)
        for i in range(1500 if n == 1 else 300):
            tq.tq_q8_attention(ctx.handle, cache, q, lens, N, workspace=ws, out=out)
            if i % 50 == 49:
                bad += (out != want).sum()
        assert int(bad) == 0


def test_a_cache_past_32_bits(ctx):
    """5.6 GB of blocks: the last sequence-head's last tokens lie past 2^32 bytes."""
    B, H, cap = 1, 8, 2_730_000
    cache = tq.Cache(ctx, B, H, cap, device=DEV)
    n = 300
    k, v = queries(1, B, H, n, BF), queries(2, B, H, n, BF)
    at = cap - n
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([at]))
    q = queries(3, B, 2 * H, 2, BF)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([cap]), cap, key_begin=ints([[at, at]]))
    kv, vv = (np64(t) for t in tq.tq_dequantize(ctx.handle, cache, at, cap))
    small = q8.Model(1, 384)  # the same tokens at the same place in their block
    small.exp[:] = q8.MIN_EXP  # a block never written: the library's zeroed scales count as the smallest
    small.append(0, at % 64, np64(k)[0, 7])
    np.testing.assert_array_equal(kv[0, 7], small.values()[0, at % 64:at % 64 + n])
    check(np64(got), np64(q), kv, vv, [n], [2], dtype=BF, out_dtype=BF)
    dst = tq.Cache(ctx, B, H, 64, device=DEV)
    w = torch.rand(B, H, cap, generator=gen(1), device=DEV)
    kept, _, _, _ = tq.tq_q8_evict(ctx.handle, cache, dst, ints([cap]), w, 64, 0, 40)
    kd, _ = tq.tq_dequantize(ctx.handle, dst, 0, 64)
    model = q8.Model(1, 64)
    rows = np.zeros((64, 128))
    for i, s in enumerate(kept[0, 7].cpu().numpy()):
        rows[i] = kv[0, 7, s - at] if s >= at else 0
    model.append(0, 0, rows)
    np.testing.assert_array_equal(np64(kd)[0, 7], model.values()[0])


def refused(status, f, *a, **kw):
    with pytest.raises(tq.TQError) as e:
        f(*a, **kw)
    assert e.value.status == status


def test_refusals(ctx):
    cache, _, _ = make(ctx, 2, 2, 128, [100, 5])
    q, lens = queries(1, 2, 4, 1, BF), ints([100, 5])
    att = tq.tq_q8_attention
    h = ctx.handle
    refused(tq.TQ_ERR_ARG, att, h, cache, queries(1, 2, 3, 1, BF), lens, 128)
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 129)
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 0)
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 128, softcap=-1.0)
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 128, scale=float("nan"))
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 128, k_positions=ints(np.zeros((2, 2, 128))))
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 128, weights_in=torch.zeros(2, 2, 128, device=DEV))
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 128, out=torch.zeros(2, 4, 1, 128, device=DEV, dtype=HF))
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 128, out=torch.zeros(2, 1, 1, 128, device=DEV, dtype=BF).expand(2, 4, 1, 128))
    refused(tq.TQ_ERR_WORKSPACE, att, h, cache, q, lens, 128, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    refused(tq.TQ_ERR_ARG, att, h, cache, q, lens, 128, out=q)
    odd = torch.zeros(2, 4, 1, 132, dtype=BF, device=DEV)[..., :128]
    refused(tq.TQ_ERR_ALIGN, att, h, cache, odd, lens, 128)
    with pytest.raises(ValueError):
        att(h, cache, q, lens.long(), 128)
    with pytest.raises(ValueError):
        att(h, cache, q, lens, 128, slopes=torch.zeros(2, device=DEV))
    other = tq.Context(128, 4, "KQV", 1)
    kqv = tq.Cache(other, 2, 2, 128, device=DEV)
    refused(tq.TQ_ERR_STATE, att, other.handle, kqv, q, lens, 128)
    other.close()
