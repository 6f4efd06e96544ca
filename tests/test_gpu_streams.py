"""Calls on a stream that is not the current one, with the tensors that the binding makes."""

import pytest
import torch

from quantised_kv_cache_gb300 import tq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantised_kv_cache_gb300 import build
    build.build()


def test_memory_of_the_current_stream_is_not_the_calls():
    """While calls run on another stream, the current one allocates, fills and drops tensors of the workspaces' and results' sizes."""
    ctx = tq.Context(128, 8, "Q8", 1)
    B, Hq, H, n, N = 2, 32, 8, 2, 20000
    g = torch.Generator(device=DEV).manual_seed(1)
    cache, dst = tq.Cache(ctx, B, H, N, device=DEV), tq.Cache(ctx, B, H, 4096, device=DEV)
    k = torch.randn(B, H, N, 128, generator=g, device=DEV).to(BF)
    tq.tq_q8_append(ctx.handle, cache, k, k, torch.zeros(B, dtype=torch.int32, device=DEV))
    q = torch.randn(B, Hq, n, 128, generator=g, device=DEV).to(BF)
    lens = torch.full((B,), N, dtype=torch.int32, device=DEV)
    pos = torch.arange(B * n, dtype=torch.int32, device=DEV).view(B, n)
    tq.tq_set_rope(ctx.handle)

    w = torch.zeros(B, H, N, device=DEV)
    x = tq.tq_rotary(ctx.handle, q, pos)
    y = tq.tq_q8_attention(ctx.handle, cache, x, lens, N, weights_in=w, weights=w)
    want = [t.clone() for t in (x, y, w, *tq.tq_q8_evict(ctx.handle, cache, dst, lens, w, 4096, 4, 64))]
    sizes = [t.numel() * t.element_size() for t in want] + [tq.tq_q8_attention_workspace(ctx.handle, B, Hq, H, n, N, weights=True)]
    side, weights = torch.cuda.Stream(), torch.zeros(B, H, N, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            weights.zero_()
        side.wait_stream(torch.cuda.current_stream())
        x = tq.tq_rotary(ctx.handle, q, pos, stream=side)
        y = tq.tq_q8_attention(ctx.handle, cache, x, lens, N, weights_in=weights, weights=weights, stream=side)
        rest = tq.tq_q8_evict(ctx.handle, cache, dst, lens, weights, 4096, 4, 64, stream=side)
        for size in sizes:
            torch.empty(size, dtype=torch.uint8, device=DEV).fill_(0xff)
        torch.cuda.synchronize()
        for got, ref in zip((x, y, weights, *rest), want):
            assert torch.equal(got, ref)
    assert tq.tq_get_device_error(ctx.handle) == 0
    ctx.close()
