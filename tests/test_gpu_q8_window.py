"""Paged 8-bit caches whose oldest blocks have been given back: a block that no query sees need not be mapped."""

import numpy as np
import pytest
import torch

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


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rows,dtype", [(1, BF), (16, HF), (40, BF), (40, HF), (8, F32), (80, F32)])
@pytest.mark.parametrize("begin", [64, 100, 127, 192, 448, 600])
def test_blocks_before_every_window_are_not_missed(rows, dtype, begin):
    """Both heads' table entries before the first seen block are -1 (one head) and past the pool (the other); the results are those of the
    whole cache, nothing is reported, and the next block that is given back is."""
    ctx = tq.Context(128, 8, "Q8", 1)
    H, N, cap = 2, 700, 704
    n = cap // 64
    g = torch.Generator(device=DEV).manual_seed(1)
    table = torch.randperm(H * n + 3, generator=g, device=DEV)[:H * n].int().view(1, H, n)
    cache = tq.PagedCache(ctx, 1, H, cap, H * n + 3, table, device=DEV)
    k, v = (torch.randn(1, H, N, 128, generator=g, device=DEV).to(BF) for _ in range(2))
    tq.tq_q8_append(ctx.handle, cache, k, v, ints([0]))
    q = torch.randn(1, H * 2, rows // 2 if rows > 1 else 1, 128, generator=g, device=DEV).to(dtype)
    if rows == 1:
        q = q[:, ::2].contiguous()
    first = begin + torch.arange(q.shape[2], device=DEV, dtype=torch.int32)[None]

    def call():
        w = torch.full((1, H, cap), 7.0, device=DEV)
        out = tq.tq_q8_attention(ctx.handle, cache, q, ints([N]), cap, key_begin=first.contiguous(), key_end=ints([[N] * q.shape[2]]), weights_in=w,
                                 weights=w)
        return out, w

    want = call()
    assert tq.tq_get_device_error(ctx.handle) == 0
    seen = begin // 64
    cache.block_table[0, 0, :seen], cache.block_table[0, 1, :seen] = -1, cache.pool_blocks
    got = call()
    assert tq.tq_get_device_error(ctx.handle) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((got[1][..., :begin] == 7).all())
    cache.block_table[0, 1, seen] = -1
    call()
    assert tq.tq_get_device_error(ctx.handle) == tq.TQ_ERR_ARG
    ctx.close()
