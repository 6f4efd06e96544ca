"""Capped scores over the 8-bit cache with caps of every size, up to those that are meant as none."""

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


@pytest.mark.parametrize("softcap", [2.0 ** -60, 0.01, 5.0, 100.0, 128.0, 129.0, 1e3, 1e4, 1e5, 1e8, 2.0 ** 39, 2.0 ** 40, 3e38])
@pytest.mark.parametrize("rows,dtype", [(16, HF), (40, HF), (40, BF), (8, F32)])
def test_caps_of_every_size(ctx, softcap, rows, dtype):
    """Scores are off by 130 U of their products' magnitudes and by 2^-21 of the cap up to 128, 2^-19 of themselves beyond; a probability by twice
    the largest of that, and by its own bits: 2^-11 (2^-8, 2^-22) and what 127 small ones of a tile may drop, 2^-21 (2^-18) of its largest each. The bound is on a row's error as a vector."""
    N = 700
    k, v = (2 * torch.randn(1, 1, N, 128, generator=gen(i), device=DEV) for i in (1, 2))
    cache = tq.Cache(ctx, 1, 1, N, device=DEV)
    tq.tq_q8_append(ctx.handle, cache, k.to(BF), v.to(BF), ints([0]))
    kv, vv = (t.double() for t in tq.tq_dequantize(ctx.handle, cache, 0, N))
    q = (1.5 * torch.randn(1, rows, 1, 128, generator=gen(3), device=DEV)).to(dtype)
    w = torch.empty(1, 1, N, device=DEV)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints([N]), N, softcap=softcap, weights=w)
    t = SCALE * torch.einsum("bhnd,bkd->bhnk", q.double(), kv[:, 0])
    e = 130 * 2.0 ** -24 * SCALE * torch.einsum("bhnd,bkd->bhnk", q.double().abs(), kv[:, 0].abs())
    e = e + (2.0 ** -21 * softcap if softcap <= 128 else 2.0 ** -19 * t.abs())
    t = softcap * torch.tanh(t / softcap)
    p = torch.softmax(t, -1)
    rel = 2 * e.amax(-1) + 2.0 ** -19
    share = {HF: 2.0 ** -11 + 2.0 ** -14, BF: 2.0 ** -8 + 2.0 ** -8, F32: 2.0 ** -22}[dtype]
    want = torch.einsum("bhnk,bkd->bhnd", p, vv[:, 0])
    mass = torch.einsum("bhnk,bk->bhn", p, vv[:, 0].norm(dim=-1))
    err = (got.double() - want).norm(dim=-1)
    tol = (rel + share + 2.0 ** -16) * mass + want.norm(dim=-1) * torch.finfo(dtype).eps / 2 * 1.01
    assert bool((err <= tol).all()), float((err / tol).max())
    bf = 2.0 ** -9 if dtype == BF else 0.0  # queries of many bf16 rows lose their smallest coordinates: 2 e of 2^-17 x 6 x 2 x 128 / 11.3
    assert bool(((w.double() - p.sum((1, 2))[:, None]).abs() <= (p * (rel[..., None] + 2.0 ** -15 + bf)).sum((1, 2))[:, None] + 1e-30).all())


def test_caps_without_a_reciprocal_are_refused(ctx):
    cache = tq.Cache(ctx, 1, 1, 64, device=DEV)
    q = torch.zeros(1, 2, 1, 128, dtype=BF, device=DEV)
    for bad in (1e-30, 1e-45, -1.0, float("inf"), float("nan")):
        with pytest.raises(tq.TQError) as e:
            tq.tq_q8_attention(ctx.handle, cache, q, ints([64]), 64, softcap=bad)
        assert e.value.status == tq.TQ_ERR_ARG
