"""One heavy key before a long tail over the 8-bit cache: the tail's probabilities are small, its mass is not.

Every bound is on a row's error as a vector. A probability p_j that enters the value sum off by d_j adds
d_j v_j to the result, so the error is at most sum_j |d_j| |v_j|, plus the rounding of the result."""

import numpy as np
import pytest
import torch

from quantised_kv_cache_gb300 import tq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SCALE = 128 ** -0.5


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


def attend(q, k, v, softcap, slopes):
    """fp64 attention of q [B][Hq][n][128] over all of k, v [B][1][N][128] (queries at the last slot), and per row sum_j p_j |v_j|."""
    t = SCALE * torch.einsum("bhnd,bkd->bhnk", q.double(), k[:, 0].double())
    if softcap:
        t = softcap * torch.tanh(t / softcap)
    if slopes is not None:
        N, n = k.shape[2], q.shape[2]
        at = torch.arange(N - n, N, device=DEV).double()
        t = t - slopes.double()[None, :, None, None] * (at[:, None] - torch.arange(N, device=DEV).double()[None]).abs()
    p = torch.softmax(t, -1)
    return torch.einsum("bhnk,bkd->bhnd", p, v[:, 0].double()), torch.einsum("bhnk,bk->bhn", p, v[:, 0].double().norm(dim=-1))


# keys, how far the heavy one's score lies above the others', ratio of neighbouring blocks' value scales
TAILS = [(8192, 10.0, 16), (32768, 10.0, 16), (32768, 11.0, 8), (131072, 13.0, 1), (131072, 13.0, 16), (131072, 15.0, 16)]


@pytest.mark.parametrize("N,gap,ratio", TAILS)
@pytest.mark.parametrize("heads,n", [(16, 1), (17, 1), (20, 15)])
@pytest.mark.parametrize("kind", ["plain", "capped", "biased"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_heavy_key_before_a_long_tail(ctx, N, gap, ratio, heads, n, kind, dtype):
    """16 rows a KV head and 17 (units of one row tile), and 300. More KV heads than SMs, all of the same tokens, so that a CTA works on most of a
    sequence by itself: the heavy key's tile is in its slice.

    A probability enters as terms of 2^8 times its ratio to the largest among 128 tokens. bf16: two e4m3 terms leave 2^-8 of numbers from 2^-2 on
    and 2^-10 (half their smallest step) of smaller ones, so |d_j| <= 2^-8 p_j or 2^-18 of the largest, 2^-14 in a block whose value scale
    is folded in at 1 : 16, and 64 such are 2^-8 of the tokens' mass. fp16: the third term, e5m2, leaves an eighth of that: 2^-11, and 2^-11 of the mass. The scores' own errors (sums of 128 products
    in fp32, queries' smallest coordinates) are below 2^-11 here. Then the rounding to the type."""
    H = torch.cuda.get_device_properties(0).multi_processor_count + 8
    rest = torch.cat([torch.zeros(1, device=DEV), torch.ones(127, device=DEV)])
    k = 0.3 * torch.randn(1, 1, N, 128, generator=gen(1), device=DEV) * rest
    k[:, :, 0] = 0.0
    k[:, :, 0, 0] = 16.0
    q = torch.randn(1, heads, n, 128, generator=gen(2), device=DEV) * rest
    q[..., 0] = gap / SCALE / 16
    v = (0.5 + torch.randn(1, 1, N, 128, generator=gen(3), device=DEV)).clamp(-3.9, 3.9)
    v[:, :, 5::64, 127] = 4.0  # every block's largest, so that neighbouring scales are exactly `ratio` apart
    v[:, :, 5::128, 127] = 4.0 * ratio
    cache = tq.Cache(ctx, 1, H, N, device=DEV)
    tq.tq_q8_append(ctx.handle, cache, k.to(BF).expand(1, H, N, 128), v.to(BF).expand(1, H, N, 128), ints([0]))
    scales = cache.tensors["v_stats"].view(F32).view(H, -1)
    assert bool((scales[:, 0::2] == ratio * scales[:, 1::2]).all())
    one = tq.Cache(ctx, 1, 1, N, device=DEV)
    tq.tq_q8_append(ctx.handle, one, k.to(BF), v.to(BF), ints([0]))
    kv, vv = tq.tq_dequantize(ctx.handle, one, 0, N)
    q = q.to(dtype)
    softcap = 60.0 if kind == "capped" else 0.0
    slopes = torch.linspace(1e-7, 1e-6, heads, device=DEV) if kind == "biased" else None
    got = tq.tq_q8_attention(ctx.handle, cache, q.repeat(1, H, 1, 1), ints([N]), N, key_end=ints(np.full((1, n), N)), softcap=softcap,
                             slopes=None if slopes is None else slopes.repeat(H))
    want, mass = attend(q, kv, vv, softcap, slopes)
    share = 2.0 ** -8 + 2.0 ** -8 if dtype == BF else 2.0 ** -11 + 2.0 ** -11
    err = (got.view(H, heads, n, 128).double() - want).norm(dim=-1)
    tol = (share + 2.0 ** -11) * mass + want.norm(dim=-1) * torch.finfo(dtype).eps / 2 * 1.01
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("rows", [16, 17, 300])
@pytest.mark.parametrize("kind", ["plain", "capped"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
def test_small_probabilities_of_large_values(ctx, rows, kind, dtype, order):
    """64 keys 14 above the 64 others of their tile, whose values are 2^20 larger: the result is the light keys'. Two value sums, each with
    its own block's largest probability as the reference, leave 2^-8 (2^-11) of every key's part."""
    N = 128
    heavy = slice(64 * order[0], 64 * order[0] + 64)
    rest = torch.cat([torch.zeros(1, device=DEV), torch.ones(127, device=DEV)])
    k = 0.3 * torch.randn(1, 1, N, 128, generator=gen(1), device=DEV) * rest
    k[:, :, heavy, 0] = 16.0
    q = torch.randn(1, rows, 1, 128, generator=gen(2), device=DEV) * rest
    q[..., 0] = 14.0 / SCALE / 16
    v = 2.0 ** 10 * (0.5 + torch.randn(1, 1, N, 128, generator=gen(3), device=DEV))
    v[:, :, heavy] *= 2.0 ** -20
    cache = tq.Cache(ctx, 1, 1, N, device=DEV)
    tq.tq_q8_append(ctx.handle, cache, k.to(BF), v.to(BF), ints([0]))
    kv, vv = tq.tq_dequantize(ctx.handle, cache, 0, N)
    q, softcap = q.to(dtype), 80.0 if kind == "capped" else 0.0
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([N]), N, softcap=softcap)
    want, mass = attend(q, kv, vv, softcap, None)
    err = (got.double() - want).norm(dim=-1)
    tol = ((2.0 ** -8 if dtype == BF else 2.0 ** -11) + 2.0 ** -11) * mass + want.norm(dim=-1) * torch.finfo(dtype).eps / 2 * 1.01 + 128 ** 0.5 * 2.0 ** -25
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_tails_around_masked_and_unmapped_blocks(ctx, dtype):
    """A tile of which a row sees one block alone, the one with the smaller value scale: it has the block's full resolution."""
    N, n = 256, 40
    k = 0.3 * torch.randn(1, 1, N, 128, generator=gen(1), device=DEV)
    v = 0.5 + torch.randn(1, 1, N, 128, generator=gen(3), device=DEV)
    v[:, :, 5::128, 127] = 60.0
    cache = tq.Cache(ctx, 1, 1, N, device=DEV)
    tq.tq_q8_append(ctx.handle, cache, k.to(BF), v.to(BF), ints([0]))
    kv, vv = tq.tq_dequantize(ctx.handle, cache, 0, N)
    q = torch.randn(1, 1, n, 128, generator=gen(2), device=DEV).to(dtype)
    begin = 64 + 192 * (torch.arange(n, device=DEV) % 2)  # the second block of the first tile, or nothing
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([N]), N, key_begin=begin.int()[None].contiguous(), key_end=ints([[128] * n]))
    want, mass = attend(q, kv[:, :, 64:128], vv[:, :, 64:128], 0.0, None)
    err = (got.double() - want).norm(dim=-1)[0, 0, ::2]
    tol = ((2.0 ** -8 if dtype == BF else 2.0 ** -11) + 2.0 ** -11) * mass + want.norm(dim=-1) * torch.finfo(dtype).eps / 2 * 1.01
    assert bool((err <= tol[0, 0, ::2]).all()) and not bool(got[0, 0, 1::2].any())
