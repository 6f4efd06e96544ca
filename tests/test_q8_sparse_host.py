"""Attention over listed blocks: what the host side refuses, on a machine without a GPU (as in test_q8_host)."""

import ctypes

import pytest
import torch

from quantised_kv_cache_gb300 import tq
from test_binding_streams import Tensor
from test_q8_blocks_host import LENS, binding, on  # noqa: F401 (binding: a fixture)
from test_q8_host import BASE, ELSEWHERE, TAKEN, S, cache, ctx  # noqa: F401 (ctx: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would be enqueued")
D = 128
LISTS = 1 << 35


def sparse(ctx, c=None, lists=LISTS, n_blocks=5, span=2, ws=1 << 42, ws_bytes=1 << 40, **kw):
    a = tq.tq_q8_attn(batch=2, heads_q=8, heads_kv=4, n_q=3, max_len=1024, q_dtype=tq.TQ_BF16, out_dtype=tq.TQ_BF16, d_q=BASE, d_out=ELSEWHERE,
                      d_seq_lens=LENS)
    n, h = kw.get("n_q", 3), kw.get("heads_q", 8)
    a.q_strides = a.out_strides = S(h * n * D, n * D, D)
    for name, value in kw.items():
        setattr(a, name, value)
    return tq.lib().tq_q8_sparse_attention(ctx, ctypes.byref(c or cache(a.batch, a.heads_kv)), bytes(a), lists, n_blocks, span, ws, ws_bytes, None)


def test_refusals(ctx):
    assert sparse(ctx) == sparse(ctx, span=100) == sparse(ctx, n_blocks=2 ** 31 - 1) == sparse(ctx, d_slopes=LENS) == TAKEN
    for kw in (dict(lists=None), dict(n_blocks=0), dict(n_blocks=-1), dict(span=0), dict(batch=0), dict(heads_q=6), dict(max_len=1025), dict(out_dtype=2),
               dict(scale=float("nan")), dict(softcap=-1.0), dict(d_k_positions=LENS), dict(ws=None), dict(d_out=None), dict(d_weights_in=LENS)):
        assert sparse(ctx, **kw) == tq.TQ_ERR_ARG, kw
    for kw in (dict(lists=LISTS + 2), dict(d_q=BASE + 4), dict(d_lse=LENS + 1)):
        assert sparse(ctx, **kw) == tq.TQ_ERR_ALIGN, kw
    assert sparse(ctx, d_weights=1 << 36) == tq.TQ_ERR_UNSUPPORTED
    assert sparse(None) == tq.TQ_ERR_ARG


def test_outputs_that_overlap(ctx):
    out, lists = 2 * 8 * 3 * D * 2, 2 * 4 * 2 * 5 * 4
    assert sparse(ctx, d_out=BASE) == sparse(ctx, d_out=LISTS) == sparse(ctx, d_lse=LISTS) == tq.TQ_ERR_ARG
    assert sparse(ctx, lists=ELSEWHERE + out) == sparse(ctx, lists=ELSEWHERE - lists) == TAKEN
    assert sparse(ctx, lists=ELSEWHERE + out - 4) == sparse(ctx, lists=ELSEWHERE - lists + 4) == tq.TQ_ERR_ARG


@pytest.mark.parametrize("B,Hq,H,n,span", [(2, 8, 4, 3, 2), (2, 32, 8, 2048, 64), (1, 32, 8, 500, 33), (1, 16, 4, 100, 7), (3, 2, 1, 700, 1000)])
def test_workspace(ctx, B, Hq, H, n, span):
    def need(*a):
        size = ctypes.c_size_t()
        assert tq.lib().tq_q8_sparse_attention_workspace(ctx, *a, ctypes.byref(size)) == 0
        return size.value

    most = need(B, Hq, H, n, span, 20)
    kw = dict(batch=B, heads_q=Hq, heads_kv=H, n_q=n, span=span)
    assert sparse(ctx, ws_bytes=most, **kw) == TAKEN
    assert sparse(ctx, ws_bytes=most - 1, **kw) == tq.TQ_ERR_WORKSPACE
    for m in {1, 2, n // 7 + 1, n // 2 + 1, n - 1} - {0}:  # what serves a call serves smaller ones of the same span
        assert need(B, Hq, H, m, span, 3) <= most and need(max(1, B - 1), Hq, H, m, span, 20) <= most
    size = ctypes.c_size_t()
    for bad in ((0, 8, 4, 1, 1, 1), (1, 7, 4, 1, 1, 1), (1, 8, 4, 0, 1, 1), (1, 8, 4, 1, 0, 1), (1, 8, 4, 1, 1, 0)):
        assert tq.lib().tq_q8_sparse_attention_workspace(ctx, *bad, ctypes.byref(size)) == tq.TQ_ERR_ARG


def test_past_what_the_kernels_count(ctx):
    c = cache(1, 1, 64)
    assert sparse(ctx, c, batch=1, heads_q=1 << 20, heads_kv=1, n_q=4096, max_len=64, d_q=1 << 44, d_out=1 << 46) == tq.TQ_ERR_UNSUPPORTED


def test_binding(binding):
    I32 = torch.int32
    lens = Tensor((2,), I32)

    def call(q=None, blocks=None, **kw):
        q = q or Tensor((2, 8, 3, 128))
        return tq.tq_q8_sparse_attention(1, binding, blocks or Tensor((2, 4, 2, 9), I32), q, lens, 128, **{"span": 2, "workspace": Tensor((64,)),
                                         "out": Tensor((2, 8, 3, 128)), **kw})

    call()
    for kw in (dict(span=0), dict(span=3), dict(blocks=Tensor((2, 4, 9), I32)), dict(blocks=Tensor((2, 4, 2, 9), torch.int64)),
               dict(blocks=on(Tensor((2, 4, 2, 9), I32), 1)), dict(workspace=on(Tensor((64,)), 1)), dict(out=on(Tensor((2, 8, 3, 128)), 1)),
               dict(out=Tensor((2, 8, 4, 128))), dict(q=on(Tensor((2, 8, 3, 128)), -1)), dict(slopes=Tensor((4,), torch.float32)),
               dict(out_dtype=torch.float32)):
        with pytest.raises(ValueError):
            call(**kw)
