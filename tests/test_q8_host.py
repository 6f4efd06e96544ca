"""The 8-bit cache's and the rotary calls' host side on a machine without a GPU: what is refused before anything is enqueued, and
what is not.

The calls take a context that lies in memory only (tq_init needs a GPU): right after the checks the library asks for the current
device, and fails (TQ_ERR_CUDA), so that a call's status tells whether its arguments were taken. Addresses are numbers; nothing
reads them."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from conftest import ROOT
from quantised_kv_cache_gb300 import tq

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would be enqueued")

SMS = 152
TAKEN = tq.TQ_ERR_CUDA


@pytest.fixture(scope="module")
def ctx(tmp_path_factory):
    cxx, cuda_inc = shutil.which("g++"), "/usr/local/cuda/include"
    if cxx is None or not os.path.isdir(cuda_inc):
        pytest.skip("needs g++ and the CUDA headers")
    from quantised_kv_cache_gb300 import build
    build.build()
    d = tmp_path_factory.mktemp("ctx")
    (d / "ctx.cpp").write_text('#include "tq_internal.h"\n'
                               'extern "C" tq_ctx *make(int scheme, int sms) {\n'
                               "  tq_ctx *c = new tq_ctx();\n"
                               "  c->d = tq::kD, c->scheme = scheme, c->bits = 8, c->num_sms = sms, c->device = -1;\n"
                               "  return c;\n}\n"
                               'extern "C" const unsigned long long *turns(const tq_ctx *c) { return c->rope.freq; }\n')
    csrc = os.path.join(ROOT, "quantised_kv_cache_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-I", csrc, "-I", os.path.join(ROOT, "include"), "-I", cuda_inc,
                    str(d / "ctx.cpp"), "-o", str(d / "ctx.so")], check=True, capture_output=True)
    L = ctypes.CDLL(str(d / "ctx.so"))
    L.make.restype, L.turns.restype = ctypes.c_void_p, ctypes.POINTER(ctypes.c_ulonglong)
    L.turns.argtypes = [ctypes.c_void_p]
    c = ctypes.c_void_p(L.make(tq.TQ_SCHEME_Q8, SMS))
    tq.tq_set_rope(c)
    c.turns = lambda: L.turns(c)
    return c


def cache(batch=2, heads=4, capacity=1024, at=1 << 40):
    c = tq.tq_cache()
    c.batch, c.heads_kv, c.capacity = batch, heads, capacity
    c.records, c.k_stats, c.v_stats = at, at + (1 << 36), at + (2 << 36)
    return c


S = tq._strides3
BASE = 1 << 20
ELSEWHERE = 1 << 34


# ------------------------------------------------------------------------------------------------ outputs that overlap

B, H, N, D = 2, 8, 16, 128
FUSED = (N * 3 * H * D, D, 3 * H * D)  # [batch][token][3 H heads][d], 2 bytes an element


def rotary(ctx, x, xs, y, ys, dtype=tq.TQ_BF16):
    return tq.lib().tq_rotary(ctx, x, S(*xs), y, S(*ys), dtype, B, H, N, 1 << 30, 0, None)


@pytest.mark.parametrize("x,xs,y,ys,want", [
    (BASE, (H * N * D, N * D, D), BASE, (H * N * D, N * D, D), TAKEN),                 # in place
    (BASE, FUSED, BASE, FUSED, TAKEN),                                                 # in place, a part of a fused projection
    (BASE, FUSED, BASE + 2 * H * D, FUSED, TAKEN),                                     # one part into another
    (BASE + 4 * H * D, FUSED, BASE, FUSED, TAKEN),
    (BASE, FUSED, BASE + 2 * (H - 1) * D, FUSED, tq.TQ_ERR_ARG),                       # parts that share a head
    (BASE, FUSED, BASE + 2 * 3 * H * D, FUSED, tq.TQ_ERR_ARG),                         # a token later
    (BASE, (H * N * D, N * D, D), BASE + 2 * D, (H * N * D, N * D, D), tq.TQ_ERR_ARG),  # a row later
    (BASE, (H * N * D, N * D, D), BASE + 2 * B * H * N * D - 16, (H * N * D, N * D, D), tq.TQ_ERR_ARG),  # the last 16 bytes
    (BASE, (H * N * D, N * D, D), BASE + 2 * B * H * N * D, (H * N * D, N * D, D), TAKEN),
    (BASE + 2 * B * H * N * D, (H * N * D, N * D, D), BASE, (H * N * D, N * D, D), TAKEN),
    (BASE, (H * N * D, N * D, D), BASE, (H * N * D, D, H * D), tq.TQ_ERR_ARG),         # in place, transposed
    (BASE, (2 * H * N * D, 2 * N * D, D), BASE + 2 * N * D, (2 * H * N * D, 2 * N * D, D), TAKEN),      # halves of every head's tokens
    (BASE, (2 * H * N * D, 2 * N * D, 2 * D), BASE + 2 * D, (2 * H * N * D, 2 * N * D, 2 * D), TAKEN),  # every other token
    (BASE, (2 * H * N * D, 2 * N * D, 2 * D), BASE + D, (2 * H * N * D, 2 * N * D, 2 * D), tq.TQ_ERR_ARG),
    (BASE + 2 * (N - 1) * D, (H * N * D, N * D, -D), BASE, (H * N * D, N * D, D), tq.TQ_ERR_ARG),       # the same rows backwards
    (BASE, (0, 0, D), BASE + 2 * N * D, (H * N * D, N * D, D), TAKEN),                 # a broadcast input before its output
    (BASE, (0, 0, D), BASE + 2 * N * D - 2 * D, (H * N * D, N * D, D), tq.TQ_ERR_ARG),
])
def test_rotary_outputs_that_overlap_their_input(ctx, x, xs, y, ys, want):
    assert rotary(ctx, x, xs, y, ys) == want


@pytest.mark.parametrize("ys", [(0, N * D, D), (H * N * D, 64, D), (H * N * D, N * D, 120), (H * N * D, N * D, -64)])
def test_targets_whose_own_rows_overlap(ctx, ys):
    assert rotary(ctx, BASE, (H * N * D, N * D, D), ELSEWHERE, ys) == tq.TQ_ERR_ARG
    assert attention(ctx, batch=B, heads_q=H, heads_kv=4, n_q=N, d_out=ELSEWHERE, out_strides=S(*ys)) == tq.TQ_ERR_ARG


def attention(ctx, c=None, ws=1 << 42, ws_bytes=1 << 40, **kw):
    a = tq.tq_q8_attn(batch=2, heads_q=8, heads_kv=4, n_q=3, max_len=1024, q_dtype=tq.TQ_BF16, out_dtype=tq.TQ_BF16, d_q=BASE, d_out=ELSEWHERE,
                      d_seq_lens=1 << 30)
    n, h = kw.get("n_q", 3), kw.get("heads_q", 8)
    a.q_strides = a.out_strides = S(h * n * D, n * D, D)
    for name, value in kw.items():
        setattr(a, name, value)
    return tq.lib().tq_q8_attention(ctx, ctypes.byref(c or cache(a.batch, a.heads_kv)), bytes(a), ws, ws_bytes, None)


def test_attention_outputs_that_overlap(ctx):
    size = 2 * 8 * 3 * D
    slots = 2 * 4 * 1024 * 4
    assert attention(ctx) == TAKEN
    for at, status in ((BASE, tq.TQ_ERR_ARG), (BASE + 2 * size - 16, tq.TQ_ERR_ARG), (BASE + 2 * size, TAKEN), (BASE - 2 * size, TAKEN),
                       (BASE - 2 * size + 16, tq.TQ_ERR_ARG)):
        assert attention(ctx, d_out=at) == status
        assert attention(ctx, d_out=at, out_dtype=tq.TQ_F32) == (TAKEN if status == TAKEN and at > BASE else tq.TQ_ERR_ARG)
    w = 1 << 36
    assert attention(ctx, d_weights=w) == TAKEN
    assert attention(ctx, d_weights=w, d_weights_in=w) == TAKEN
    assert attention(ctx, d_weights=w, d_weights_in=w + slots) == TAKEN
    assert attention(ctx, d_weights=w, d_weights_in=w + 4) == tq.TQ_ERR_ARG
    assert attention(ctx, d_weights=w, d_weights_in=w - slots + 4) == tq.TQ_ERR_ARG
    assert attention(ctx, d_weights=w, d_lse=w + slots) == TAKEN
    assert attention(ctx, d_weights=w, d_lse=w + slots - 4) == tq.TQ_ERR_ARG
    assert attention(ctx, d_weights=w, d_lse=ELSEWHERE + 2 * size - 4) == tq.TQ_ERR_ARG
    assert attention(ctx, d_weights=BASE + 2 * size - 4) == tq.TQ_ERR_ARG


def evict(ctx, **kw):
    a = dict(lens=1 << 30, weights=1 << 31, positions=1 << 32, kept=1 << 33, dst_lens=ELSEWHERE, dst_weights=1 << 35, dst_positions=1 << 36)
    a.update(kw)
    src, dst = cache(2, 4, 1024), cache(2, 4, 512, at=1 << 44)
    return tq.lib().tq_q8_evict(ctx, ctypes.byref(src), ctypes.byref(dst), 2, 4, a["lens"], a["weights"], 256, 4, 16, a["positions"], a["kept"],
                                a["dst_lens"], a["dst_weights"], a["dst_positions"], None)


def test_eviction_outputs_that_overlap(ctx):
    from_, to, kept = 2 * 4 * 1024 * 4, 2 * 4 * 512 * 4, 2 * 4 * 256 * 4
    assert evict(ctx) == TAKEN
    assert evict(ctx, dst_lens=1 << 30) == TAKEN  # the lengths' own place
    assert evict(ctx, dst_lens=(1 << 30) + 4) == tq.TQ_ERR_ARG
    for out, size in (("dst_weights", to), ("dst_positions", to), ("kept", kept)):
        for src, bytes_ in (("weights", from_), ("positions", from_), ("lens", 8)):
            at = dict(lens=1 << 30, weights=1 << 31, positions=1 << 32)[src]
            assert evict(ctx, **{out: at}) == tq.TQ_ERR_ARG
            assert evict(ctx, **{out: at + bytes_ - 4}) == tq.TQ_ERR_ARG
            assert evict(ctx, **{out: at - size + 4}) == tq.TQ_ERR_ARG
            assert evict(ctx, **{out: at + bytes_}) == TAKEN and evict(ctx, **{out: at - size}) == TAKEN
    assert evict(ctx, dst_weights=1 << 36) == tq.TQ_ERR_ARG
    assert evict(ctx, kept=(1 << 35) + to - 4) == tq.TQ_ERR_ARG
    assert evict(ctx, dst_positions=(1 << 33) + kept - 4) == tq.TQ_ERR_ARG
    assert evict(ctx, dst_lens=(1 << 33) + 4) == tq.TQ_ERR_ARG
    assert evict(ctx, positions=None, dst_weights=None, dst_positions=None) == TAKEN


# ------------------------------------------------------------------------------------------------ workspaces

def size(ctx, n_q, max_len, batch=8, heads_q=32, heads_kv=8, weights=1):
    out = ctypes.c_size_t()
    assert tq.lib().tq_q8_attention_workspace(ctx, batch, heads_q, heads_kv, n_q, max_len, weights, ctypes.byref(out)) == tq.TQ_OK
    return out.value


def fits(ctx, ws, n_q, max_len, batch=8, heads_q=32, heads_kv=8, weights=1, out_dtype=tq.TQ_BF16):
    w = dict(d_weights=1 << 45) if weights else {}
    return attention(ctx, cache(batch, heads_kv, max(max_len, 1 << 19)), ws_bytes=ws, batch=batch, heads_q=heads_q, heads_kv=heads_kv, n_q=n_q,
                     max_len=max_len, out_dtype=out_dtype, d_out=1 << 46, **w)


@pytest.mark.parametrize("weights", [0, 1])
def test_a_larger_calls_workspace_serves_the_smaller_ones(ctx, weights):
    """Every size below, in each of sequences, query tokens and slots, whatever the results' type."""
    sizes = [(b, n, m) for b in (1, 3, 16) for n in (1, 2, 4, 5, 8, 16, 17, 40, 512, 2048)
             for m in (1, 1000, 9728, 9984, 19456, 100000, 131072, 524288)]
    for big in [(16, 2048, 524288), (16, 17, 524288), (3, 512, 19456), (16, 40, 9984), (3, 4, 131072), (1, 16, 100000)]:
        ws = size(ctx, big[1], big[2], big[0], weights=weights)
        assert fits(ctx, ws, big[1], big[2], big[0], weights=weights) == TAKEN
        for b, n, m in sizes:
            if b <= big[0] and n <= big[1] and m <= big[2]:
                for dt in (tq.TQ_BF16, tq.TQ_F32):
                    assert fits(ctx, ws, n, m, b, weights=weights, out_dtype=dt) == TAKEN, (big, b, n, m, dt)
                assert fits(ctx, ws, n, m, b, weights=0) == TAKEN


def test_workspaces_of_long_and_of_many_row_calls(ctx):
    ws = size(ctx, 512, 131072, 8)
    assert fits(ctx, ws, 1, 131072, 8) == TAKEN
    ws = size(ctx, 1, 524416, 16)
    assert fits(ctx, ws, 1, 524288, 16) == TAKEN


def test_no_room_for_scores_that_are_not_kept(ctx):
    """17 to 64 rows with 16-bit results: their scores are formed again, and a sizing call that says so has no room for them."""
    scores = 32 * 16 * 131072 * 4
    both, half = size(ctx, 16, 131072, 1, weights=1), size(ctx, 16, 131072, 1, weights=2)
    assert both > scores and half < scores // 4
    assert fits(ctx, half, 16, 131072, 1) == TAKEN
    assert size(ctx, 4, 131072, 1, weights=2) == size(ctx, 4, 131072, 1, weights=1) > 32 * 4 * 131072 * 4  # up to 16 rows they are kept
    for bad in (-1, 3):
        out = ctypes.c_size_t()
        assert tq.lib().tq_q8_attention_workspace(ctx, 1, 8, 8, 1, 100, bad, ctypes.byref(out)) == tq.TQ_ERR_ARG


@pytest.mark.parametrize("n_q", [1, 4, 17, 300])
def test_workspaces_that_are_too_small_are_refused(ctx, n_q):
    for weights in (0, 1):
        ws = size(ctx, n_q, 5000, weights=weights)
        assert fits(ctx, ws, n_q, 5000, weights=weights) == TAKEN
        assert fits(ctx, 2_000_000, n_q, 5000, weights=weights) == tq.TQ_ERR_WORKSPACE  # below the partial records alone


# ------------------------------------------------------------------------------------------------ frequencies

def exact_turns(dim, base=10000.0, factor=1.0, original_len=0.0, low=0.0, high=0.0):
    """2^64 f_i / (2 pi) in 60 decimal digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    base, factor, original_len, low, high = (Decimal(x) for x in (base, factor, original_len, low, high))
    out = []
    for i in range(dim // 2):
        f = (-(Decimal(2 * i) / dim) * base.ln()).exp()
        if factor > 1:
            keep = Decimal(0)
            if low or high:
                keep = min(max((original_len * f / two_pi - low) / (high - low), Decimal(0)), Decimal(1))
            f = (1 - keep) * f / factor + keep * f
        out.append(f / two_pi * 2 ** 64)
    return out


@pytest.mark.parametrize("kw", [dict(dim=128), dict(dim=64, base=500000.0), dict(dim=72, base=1e6), dict(dim=8, base=1.0000001), dict(dim=128, base=1e300),
                                dict(dim=128, base=37.3, factor=7.3), dict(dim=128, base=500000.0, factor=8.0, original_len=8192.0, low=1.0, high=4.0),
                                dict(dim=96, base=1e4, factor=31.7, original_len=4096.5, low=0.7, high=32.1),
                                dict(dim=64, factor=2.0, original_len=1e308, low=0.0, high=1e-300)], ids=str)
def test_frequencies_to_the_last_of_64_bits(ctx, kw):
    """A position turns by its multiple of the frequency, so that an error of the frequency grows to 2^31 times itself: it is half a unit
    of 2^-64 turns (and what 106-bit arithmetic leaves), 2^-34 turns at the farthest position."""
    tq.tq_set_rope(ctx, **kw)
    turns = ctx.turns()
    for i, want in enumerate(exact_turns(**kw)):
        assert abs(int(turns[i]) - want) <= 0.51, (i, float(int(turns[i]) - want))


# ------------------------------------------------------------------------------------------------ nothing to do

def test_calls_of_no_tokens_need_no_vectors(ctx):
    """A tensor without elements has no address. (As they have nothing to enqueue the calls end at the device's check.)"""
    L, s = tq.lib(), S(0, 0, 0)
    c = ctypes.byref(cache())
    assert L.tq_rotary(ctx, None, s, None, s, tq.TQ_BF16, 2, 4, 0, None, 0, None) == TAKEN
    assert L.tq_q8_append(ctx, c, None, s, None, s, tq.TQ_BF16, 2, 4, 0, 1 << 30, None, 0, None, None) == TAKEN
    assert L.tq_append_quantize(ctx, c, None, None, tq.TQ_BF16, 2, 4, 0, 1 << 30, None) == tq.TQ_OK
    # with tokens they do
    assert L.tq_rotary(ctx, None, s, ELSEWHERE, s, tq.TQ_BF16, 1, 1, 1, 1 << 30, 0, None) == tq.TQ_ERR_ARG
    assert L.tq_rotary(ctx, BASE, s, ELSEWHERE, s, tq.TQ_BF16, 1, 1, 1, None, 0, None) == tq.TQ_ERR_ARG
    assert L.tq_q8_append(ctx, c, BASE, s, None, s, tq.TQ_BF16, 2, 4, 1, 1 << 30, None, 0, None, None) == tq.TQ_ERR_ARG
    # and other arguments are checked all the same
    assert L.tq_rotary(ctx, None, s, None, s, 7, 2, 4, 0, None, 0, None) == tq.TQ_ERR_ARG
    assert L.tq_q8_append(ctx, c, None, s, None, s, tq.TQ_BF16, 2, 4, 0, None, None, 0, None, None) == tq.TQ_ERR_ARG


# ------------------------------------------------------------------------------------------------ sizes past the kernels' indices

def test_sizes_that_no_launch_or_index_holds_are_refused_before_anything_runs(ctx):
    big = dict(ws_bytes=1 << 62)
    for kw in (dict(batch=65536, heads_q=1, heads_kv=1, n_q=1), dict(batch=1, heads_q=65536, heads_kv=65536, n_q=1)):
        c = cache(kw["batch"], kw["heads_kv"])
        assert attention(ctx, c, d_out=1 << 50, **kw, **big) == TAKEN
        assert attention(ctx, c, d_out=1 << 50, d_weights=1 << 52, **kw, **big) == tq.TQ_ERR_UNSUPPORTED
    # rows of a KV head, and units x tiles, in 32 bits
    most = 2 ** 31 - 1024
    long = cache(1, 1, most)
    assert attention(ctx, long, batch=1, heads_q=1, heads_kv=1, n_q=1, max_len=most, **big) == TAKEN
    assert attention(ctx, cache(1, 1), batch=1, heads_q=64, heads_kv=1, n_q=1 << 26, d_out=1 << 60, **big) == tq.TQ_ERR_UNSUPPORTED
    assert attention(ctx, long, batch=1, heads_q=1, heads_kv=1, n_q=129 * 256, max_len=most, **big) == tq.TQ_ERR_UNSUPPORTED
    assert attention(ctx, long, batch=1, heads_q=1, heads_kv=1, n_q=128 * 256, max_len=most, **big) == TAKEN
    # slots whose block or tile ends past 2^31
    for capacity, want in ((most, TAKEN), (most + 1, tq.TQ_ERR_UNSUPPORTED), (2 ** 31 - 1, tq.TQ_ERR_UNSUPPORTED)):
        c = cache(1, 1, capacity)
        assert attention(ctx, c, batch=1, heads_q=1, heads_kv=1, n_q=1, max_len=64) == want
        assert tq.lib().tq_q8_append(ctx, ctypes.byref(c), BASE, S(0, 0, 0), BASE, S(0, 0, 0), tq.TQ_BF16, 1, 1, 1, 1 << 30, None, 0, None, None) == want
        out = tq.tq_cache_sizes()
        assert tq.lib().tq_cache_sizes_get(ctx, 1, 1, capacity, ctypes.byref(out)) == (tq.TQ_OK if want == TAKEN else want)


# ------------------------------------------------------------------------------------------------ alignment

def test_alignment_of_every_pointer(ctx):
    """Vectors, planes and workspaces: 16 bytes. Numbers of 4 bytes: their own size."""
    L = tq.lib()
    rows = S(H * N * D, N * D, D)
    assert rotary(ctx, BASE + 8, rows, ELSEWHERE, rows) == tq.TQ_ERR_ALIGN
    assert rotary(ctx, BASE, rows, ELSEWHERE + 2, rows) == tq.TQ_ERR_ALIGN
    for at, want in (((1 << 30) + 2, tq.TQ_ERR_ALIGN), ((1 << 30) + 4, TAKEN)):
        assert L.tq_rotary(ctx, BASE, rows, ELSEWHERE, rows, tq.TQ_BF16, B, H, N, at, 0, None) == want
        kv = S(4 * N * D, N * D, D)

        def append(lens=1 << 30, new=None, pos=None):
            return L.tq_q8_append(ctx, ctypes.byref(cache()), BASE, kv, BASE, kv, tq.TQ_BF16, 2, 4, N, lens, new, 1, pos, None)

        assert append(lens=at) == append(new=at) == append(pos=at) == want
        for name in ("d_seq_lens", "d_new_lens", "d_slopes", "d_key_begin", "d_key_end", "d_q_positions", "d_weights", "d_lse"):
            assert attention(ctx, **{name: at}) == want, name
        assert attention(ctx, d_weights=1 << 50, d_weights_in=at) == want
        assert attention(ctx, d_q_positions=1 << 50, d_k_positions=at) == want
        paged = cache()
        paged.block_table, paged.pool_blocks = at, 100
        assert attention(ctx, paged) == want
        for name in ("lens", "weights", "positions", "kept", "dst_lens", "dst_weights", "dst_positions"):
            assert evict(ctx, **{name: at + (1 << 48)}) == want, name
