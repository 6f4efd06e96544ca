"""Workspaces of other sizes than a call's own: larger calls' ones, and ones without room for the scores."""

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


@pytest.fixture()
def ctx():
    c = tq.Context(128, 8, "Q8", 1)
    yield c
    assert tq.tq_get_device_error(c.handle) == 0
    c.close()


@pytest.mark.parametrize("B,Hq,H,n,lens,dtype", [(2, 8, 2, 1, [3000, 100], BF), (1, 16, 4, 4, [5000], HF), (2, 8, 2, 8, [900, 1], F32), (1, 8, 2, 40, [2000], F32),
                                                 (3, 8, 2, 5, [700, 0, 4000], BF), (2, 16, 2, 100, [3000, 200], BF), (1, 8, 1, 300, [1500], HF)])
def test_weights_in_workspaces_of_every_size(ctx, B, Hq, H, n, lens, dtype):
    """The least that is taken (found byte by byte down from the sizing call's in steps of 16), the call's own, a longer call's: the same results, the
    weights up to the rounding of scores that are formed again: both are within the exponentials' 2^-19 of the same fp32 scores, whose sums
    may differ by their order (130 U of the products' magnitudes, twice)."""
    cap = 5120
    g = torch.Generator(device=DEV).manual_seed(1)
    cache = tq.Cache(ctx, B, H, cap, device=DEV)
    k, v = (torch.randn(B, H, max(lens), 128, generator=g, device=DEV).to(BF) for _ in range(2))
    new = torch.tensor(lens, dtype=torch.int32, device=DEV)
    tq.tq_q8_append(ctx.handle, cache, k, v, torch.zeros_like(new), new_lens=new)
    q = torch.randn(B, Hq, n, 128, generator=g, device=DEV).to(dtype)
    own = tq.tq_q8_attention_workspace(ctx.handle, B, Hq, H, n, cap, True, dtype)
    longer = tq.tq_q8_attention_workspace(ctx.handle, B + 2, Hq, H, n + 300, 100000, True)
    rows = torch.minimum(new, torch.full_like(new, n))

    def call(size):
        room = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
        out, w = torch.zeros_like(q), torch.empty(B, H, cap, device=DEV)
        tq.tq_q8_attention(ctx.handle, cache, q, new, cap, new_lens=rows, weights=w, workspace=room[4096:4096 + size], out=out)
        assert bool((room[:4096] == 0xA5).all()) and bool((room[4096 + size:] == 0xA5).all())
        return out, w

    out, w = call(own)
    low, high = 0, own // 16
    while high - low > 1:  # the least size in steps of 16 bytes
        mid = (low + high) // 2
        try:
            call(16 * mid)
            high = mid
        except tq.TQError as e:
            assert e.status == tq.TQ_ERR_WORKSPACE
            low = mid
    score = 130 * 2.0 ** -24 * 128 ** -0.5 * float(q.float().norm(dim=-1).max()) * float(k.float().norm(dim=-1).max())
    for size in (16 * high, longer):
        again, w2 = call(size)
        assert torch.equal(again, out)
        assert bool(((w2 - w).abs() <= w * (4 * score + 2.0 ** -18) + 1e-30).all())
    assert abs(float(w.double().sum()) / float(rows.sum() * Hq) - 1) < 1e-4
