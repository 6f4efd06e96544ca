"""Attention behind a shared prefix: what the host side refuses, on a machine without a GPU (as in test_q8_host)."""

import ctypes

import pytest
import torch

from quantised_kv_cache_gb300 import tq
from test_binding_streams import Tensor
from test_q8_blocks_host import LENS, binding, on  # noqa: F401 (binding: a fixture)
from test_q8_host import BASE, ELSEWHERE, TAKEN, S, cache, ctx  # noqa: F401 (ctx: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would be enqueued")
D = 128
PREFIX_LENS = 1 << 35


def shared(ctx, pre=None, c=None, lens=PREFIX_LENS, most=500, ws=1 << 42, ws_bytes=1 << 50, **kw):
    a = tq.tq_q8_attn(batch=2, heads_q=8, heads_kv=4, n_q=3, max_len=1024, q_dtype=tq.TQ_BF16, out_dtype=tq.TQ_BF16, d_q=BASE, d_out=ELSEWHERE,
                      d_seq_lens=LENS)
    n, h = kw.get("n_q", 3), kw.get("heads_q", 8)
    a.q_strides = a.out_strides = S(h * n * D, n * D, D)
    for name, value in kw.items():
        setattr(a, name, value)
    pre = pre or cache(1, a.heads_kv, 512, at=1 << 43)
    return tq.lib().tq_q8_shared_attention(ctx, ctypes.byref(pre), lens, most, ctypes.byref(c or cache(a.batch, a.heads_kv)), bytes(a), ws, ws_bytes,
                                           None)


def test_refusals(ctx):
    assert shared(ctx) == shared(ctx, d_slopes=LENS, d_key_begin=LENS, d_key_end=LENS, d_lse=1 << 36) == TAKEN
    for kw in (dict(lens=None), dict(most=0), dict(most=-1), dict(most=513), dict(pre=cache(2, 4, 512)), dict(pre=cache(1, 3, 512)), dict(max_len=1025),
               dict(heads_q=7), dict(n_q=0), dict(ws=None), dict(d_k_positions=LENS), dict(d_weights_in=LENS), dict(scale=float("inf"))):
        assert shared(ctx, **kw) == tq.TQ_ERR_ARG, kw
    bad = cache(1, 4, 512, at=(1 << 43) + 8)
    for kw in (dict(lens=PREFIX_LENS + 2), dict(pre=bad), dict(d_out=ELSEWHERE + 8), dict(ws=(1 << 42) + 8)):
        assert shared(ctx, **kw) == tq.TQ_ERR_ALIGN, kw
    for kw in (dict(d_weights=1 << 36), dict(d_q_positions=LENS), dict(d_q_positions=LENS, d_k_positions=LENS)):
        assert shared(ctx, **kw) == tq.TQ_ERR_UNSUPPORTED, kw
    assert shared(None) == tq.TQ_ERR_ARG


def test_outputs_that_overlap(ctx):
    out = 2 * 8 * 3 * D * 2
    assert shared(ctx, d_out=BASE) == shared(ctx, d_out=PREFIX_LENS) == shared(ctx, d_lse=PREFIX_LENS) == tq.TQ_ERR_ARG
    assert shared(ctx, lens=ELSEWHERE + out) == shared(ctx, lens=ELSEWHERE - 8) == TAKEN
    assert shared(ctx, lens=ELSEWHERE + out - 4) == shared(ctx, lens=ELSEWHERE - 4) == tq.TQ_ERR_ARG


@pytest.mark.parametrize("B,Hq,H,n", [(1, 1, 1, 1), (2, 8, 4, 3), (4, 4, 4, 4), (64, 32, 8, 1), (4, 32, 8, 512), (300, 3, 1, 7)])
def test_workspace(ctx, B, Hq, H, n):
    def need(*a):
        size = ctypes.c_size_t()
        assert tq.lib().tq_q8_shared_attention_workspace(ctx, *a, ctypes.byref(size)) == 0
        return size.value

    most = need(B, Hq, H, n, 500, 1024)
    kw = dict(batch=B, heads_q=Hq, heads_kv=H, n_q=n)
    assert shared(ctx, ws_bytes=most, **kw) == TAKEN
    assert shared(ctx, ws_bytes=most - 1, **kw) == tq.TQ_ERR_WORKSPACE
    for b in {1, B // 2 + 1, B}:
        for m in {1, n // 2 + 1, n}:
            assert need(min(b, B), Hq, H, min(m, n), 1, 1) <= most
    size = ctypes.c_size_t()
    for bad in ((0, 8, 4, 1, 1, 1), (1, 7, 4, 1, 1, 1), (1, 8, 4, 0, 1, 1), (1, 8, 4, 1, 0, 1), (1, 8, 4, 1, 1, 0)):
        assert tq.lib().tq_q8_shared_attention_workspace(ctx, *bad, ctypes.byref(size)) == tq.TQ_ERR_ARG


def test_past_what_the_kernels_count(ctx):
    big = dict(d_q=1 << 44, d_out=1 << 46)
    assert shared(ctx, c=cache(1 << 16, 1, 64), batch=1 << 16, heads_q=64, heads_kv=1, n_q=512, max_len=64, **big) == tq.TQ_ERR_UNSUPPORTED  # rows
    most = 2 ** 31 - 1024
    pre, own = cache(1, 4, most, at=1 << 43), cache(2, 4, most, at=1 << 45)
    assert shared(ctx, pre=pre, c=own, n_q=1, most=most, max_len=1) == tq.TQ_ERR_UNSUPPORTED  # slots
    assert shared(ctx, pre=pre, c=own, n_q=1, most=most - 64, max_len=64) == TAKEN


def test_binding(binding):
    I32 = torch.int32
    lens = Tensor((2,), I32)

    def call(q=None, prefix=binding, prefix_lens=lens, **kw):
        return tq.tq_q8_shared_attention(1, prefix, prefix_lens, 100, binding, q or Tensor((2, 8, 3, 128)), lens, 128,
                                         **{"workspace": Tensor((64,)), "out": Tensor((2, 8, 3, 128)), **kw})

    call()
    elsewhere = type(binding)()
    elsewhere.device_index = 1
    for kw in (dict(prefix=elsewhere), dict(prefix_lens=Tensor((1,), I32)), dict(prefix_lens=on(Tensor((2,), I32), -1)),
               dict(prefix_lens=Tensor((2,), torch.int64)), dict(q=Tensor((3, 8, 3, 128))), dict(workspace=on(Tensor((64,)), 1)),
               dict(key_begin=Tensor((2, 2), I32)), dict(lse=Tensor((2, 4, 3), torch.float32))):
        with pytest.raises(ValueError):
            call(**kw)
