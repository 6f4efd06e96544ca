"""Key bounds, choice of blocks: what the host side refuses, on a machine without a GPU (as in test_q8_host: a call that is taken
fails with TQ_ERR_CUDA where it asks for the device)."""

import ctypes

import pytest
import torch

from quantised_kv_cache_gb300 import tq
from test_binding_streams import Cache as StandIn, Library, Tensor
from test_q8_host import BASE, ELSEWHERE, TAKEN, S, cache, ctx  # noqa: F401 (ctx: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would be enqueued")
D = 128
LENS = 1 << 30


def bounds(ctx, c=None, batch=2, heads=4, n_new=3, lens=LENS, new=None, at=ELSEWHERE):
    return tq.lib().tq_q8_bounds(ctx, ctypes.byref(c or cache()), batch, heads, n_new, lens, new, at, None)


def test_bounds_refusals(ctx):
    assert bounds(ctx) == TAKEN and bounds(ctx, new=LENS + 64) == TAKEN and bounds(ctx, n_new=0) == TAKEN
    assert bounds(None) == bounds(ctx, lens=None) == bounds(ctx, at=None) == bounds(ctx, n_new=-1) == tq.TQ_ERR_ARG
    assert bounds(ctx, batch=3) == bounds(ctx, heads=5) == bounds(ctx, batch=0) == tq.TQ_ERR_ARG
    for kw in (dict(at=ELSEWHERE + 8), dict(lens=LENS + 2), dict(new=LENS + 1)):
        assert bounds(ctx, **kw) == tq.TQ_ERR_ALIGN
    size = 2 * 4 * 16 * 256
    assert bounds(ctx, at=LENS - size) == TAKEN
    assert bounds(ctx, at=LENS - size + 16) == bounds(ctx, at=LENS) == tq.TQ_ERR_ARG
    assert bounds(ctx, new=ELSEWHERE + size - 4) == tq.TQ_ERR_ARG and bounds(ctx, new=ELSEWHERE + size) == TAKEN
    assert bounds(ctx, at=(1 << 40) + 4096) == tq.TQ_ERR_ARG  # within the cache's records


def pick(ctx, c=None, ws=1 << 42, ws_bytes=1 << 40, **kw):
    a = tq.tq_q8_pick(batch=2, heads_q=8, heads_kv=4, n_q=3, span=2, max_len=1024, keep=5, sink=1, recent=2, q_dtype=tq.TQ_BF16, d_q=BASE,
                      d_seq_lens=LENS, d_bounds=1 << 33, d_blocks=ELSEWHERE)
    for name, value in kw.items():
        setattr(a, name, value)
    n, h = max(a.n_q, 1), max(a.heads_q, 1)
    if "q_strides" not in kw:
        a.q_strides = S(h * n * D, n * D, D)
    return tq.lib().tq_q8_select(ctx, ctypes.byref(c or cache()), bytes(a), ws, ws_bytes, None)


def test_choice_refusals(ctx):
    assert pick(ctx) == pick(ctx, ws=None, ws_bytes=0) == pick(ctx, span=100) == TAKEN
    for kw in (dict(batch=0), dict(heads_q=7), dict(heads_q=0), dict(heads_kv=3), dict(n_q=0), dict(span=0), dict(max_len=0), dict(max_len=1025),
               dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=3, recent=3), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(q_dtype=7),
               dict(d_q=None), dict(d_seq_lens=None), dict(d_bounds=None), dict(d_blocks=None)):
        assert pick(ctx, **kw) == tq.TQ_ERR_ARG, kw
    for kw in (dict(d_q=BASE + 8), dict(d_bounds=BASE + 4), dict(d_blocks=ELSEWHERE + 2), dict(d_seq_lens=LENS + 1), dict(d_new_lens=LENS + 3),
               dict(d_key_begin=LENS + 2), dict(d_key_end=LENS + 2), dict(q_strides=S(1024, 132, 4)), dict(ws=(1 << 42) + 4)):
        assert pick(ctx, **kw) == tq.TQ_ERR_ALIGN, kw
    assert pick(None) == tq.TQ_ERR_ARG
    assert tq.lib().tq_q8_select(ctx, None, bytes(tq.tq_q8_pick()), None, 0, None) == tq.TQ_ERR_ARG


def test_lists_that_overlap_what_is_read(ctx):
    lists = 2 * 4 * 2 * 5 * 4
    assert pick(ctx, d_blocks=BASE) == pick(ctx, d_blocks=BASE - lists + 4) == tq.TQ_ERR_ARG
    assert pick(ctx, d_blocks=BASE - lists) == TAKEN
    assert pick(ctx, d_blocks=(1 << 33) + 4096) == pick(ctx, d_blocks=LENS) == pick(ctx, d_blocks=LENS - lists + 4) == tq.TQ_ERR_ARG
    for name in ("d_new_lens", "d_key_begin", "d_key_end"):
        assert pick(ctx, **{name: ELSEWHERE + lists - 4}) == tq.TQ_ERR_ARG
        assert pick(ctx, **{name: ELSEWHERE + lists}) == TAKEN


def test_choice_workspace(ctx):
    def need(*a):
        out = ctypes.c_size_t()
        assert tq.lib().tq_q8_select_workspace(ctx, *a, ctypes.byref(out)) == 0
        return out.value

    small = need(2, 8, 4, 1, 1, 100000)
    big = need(2, 8, 4, 1, 1, 64 * 40000)
    assert small <= big and big >= 2 * 4 * 40000 * 4
    c = cache(2, 4, 64 * 40000)
    assert pick(ctx, c, n_q=1, span=1, max_len=64 * 40000, ws_bytes=big) == TAKEN
    assert pick(ctx, c, n_q=1, span=1, max_len=64 * 40000, ws_bytes=big - 1) == tq.TQ_ERR_WORKSPACE
    assert pick(ctx, c, n_q=1, span=1, max_len=64 * 40000, ws=None) == tq.TQ_ERR_WORKSPACE
    out = ctypes.c_size_t()
    for bad in ((0, 8, 4, 1, 1, 64), (1, 7, 4, 1, 1, 64), (1, 8, 4, 0, 1, 64), (1, 8, 4, 1, 0, 64), (1, 8, 4, 1, 1, 0)):
        assert tq.lib().tq_q8_select_workspace(ctx, *bad, ctypes.byref(out)) == tq.TQ_ERR_ARG


def test_choice_past_what_the_kernels_count(ctx):
    c = cache(1, 1, 64)
    assert pick(ctx, c, batch=1, heads_q=1 << 20, heads_kv=1, n_q=4096, max_len=64, span=4096) == tq.TQ_ERR_UNSUPPORTED  # rows of a KV head
    c = cache(1 << 16, 64, 64)
    assert pick(ctx, c, batch=1 << 16, heads_q=64, heads_kv=64, n_q=128, span=1, max_len=64) == tq.TQ_ERR_UNSUPPORTED  # lists


def test_the_packed_choice_is_the_struct():
    names = [n for n, _ in tq.tq_q8_pick._fields_]
    values, want = [], {}
    for k, name in enumerate(names):
        got = [100 + k + i for i in range(3 if name == "q_strides" else 1)]
        values += got
        want[name] = got
    raw = tq._pack_pick.pack(*values)
    assert len(raw) == ctypes.sizeof(tq.tq_q8_pick)
    a = tq.tq_q8_pick.from_buffer_copy(raw)
    assert {n: list(getattr(a, n)) if n == "q_strides" else [getattr(a, n)] for n in names} == want


# ------------------------------------------------------------------------------------------------ the binding

@pytest.fixture()
def binding(monkeypatch):
    monkeypatch.setattr(tq, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7, raising=False)
    c = StandIn()
    c.bounds_blocks = 16
    return c


def on(tensor, index):
    tensor.get_device = lambda: index
    return tensor


def test_binding_wants_the_cache_s_arrays(binding):
    I32, I8 = torch.int32, torch.int8
    lens, ok = Tensor((2,), I32), Tensor((16, 2, 128), I8)
    assert tq.tq_q8_bounds(1, binding, ok, lens, 3) is ok
    for bad in (Tensor((15, 2, 128), I8), Tensor((16, 2, 128), torch.uint8), on(Tensor((16, 2, 128), I8), 1)):
        with pytest.raises(ValueError):
            tq.tq_q8_bounds(1, binding, bad, lens, 3)
        with pytest.raises(ValueError):
            tq.tq_q8_select(1, binding, bad, Tensor((2, 8, 3, 128)), lens, 128, 4, blocks=Tensor((2, 4, 3, 4), I32), workspace=Tensor((64,)))
    with pytest.raises(ValueError):
        tq.tq_q8_bounds(1, binding, ok, Tensor((3,), I32), 3)

    def select(q=None, **kw):
        kw = {"blocks": Tensor((2, 4, 2, 4), I32), "workspace": Tensor((64,)), "span": 2, **kw}
        return tq.tq_q8_select(1, binding, ok, q or Tensor((2, 8, 3, 128)), lens, 128, 4, **kw)

    select()
    for kw in (dict(blocks=Tensor((2, 4, 3, 4), I32)), dict(span=0), dict(workspace=on(Tensor((64,)), -1)), dict(key_begin=Tensor((2, 4), I32)),
               dict(new_lens=Tensor((2,), torch.int64)), dict(q=on(Tensor((2, 8, 3, 128)), 1))):
        with pytest.raises(ValueError):
            select(**kw)
    with pytest.raises(ValueError):  # a query for each of two sequences, but lengths of one
        tq.tq_q8_select(1, binding, ok, Tensor((1, 8, 3, 128)), lens, 128, 4, blocks=Tensor((1, 4, 3, 4), I32), workspace=Tensor((64,)))
