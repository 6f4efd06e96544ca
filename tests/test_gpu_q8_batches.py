"""Batches of more sequences than one pass of the planning takes, sequences that share blocks, and a general step as a graph."""

import numpy as np
import pytest
import torch

from quantised_kv_cache_gb300 import tq
from test_gpu_q8_attention import BF, DEV, F32, HF, check, ctx, gen, ints, make, np64, queries, _built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq,H,n,longest", [(1100, 4, 1, 5, 300), (2500, 18, 1, 1, 70), (1030, 4, 1, 50, 130), (9000, 20, 1, 1, 20)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompts_of_many_sequences(ctx, B, Hq, H, n, longest, dtype):
    """Units of one row tile and of two, more than 1024 and more than 8192 of them; some sequences are empty, some bring no query tokens."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, longest + 1, B)
    lens[0] = longest
    new = np.minimum(rng.integers(0, n + 1, B), lens)
    cache, k, v = make(ctx, B, H, longest + 3, lens, seed=3, paged=True)
    q = queries(5, B, Hq, n, dtype, "tokens")
    out, lse, w = torch.full_like(q, 77.0), torch.zeros(B, Hq, n, device=DEV), torch.zeros(B, H, longest + 3, device=DEV)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), longest + 3, new_lens=ints(new), out=out, lse=lse, weights_in=w, weights=w)
    some = sorted({0, B - 1, *rng.integers(0, B, 60).tolist()})
    check(np64(got[some]), np64(q[some]), k[some], v[some], lens[some], new[some], dtype=dtype, out_dtype=dtype, lse=np64(lse[some]), weights=np64(w[some]))
    late = torch.arange(n, device=DEV)[None] >= torch.as_tensor(new, device=DEV)[:, None]
    assert bool((got.transpose(1, 2)[late] == 77).all())
    live = torch.as_tensor(new, device=DEV).double() * Hq
    assert bool(((w.double().sum((1, 2)) - live).abs() <= 1e-4 * live).all())


@pytest.mark.parametrize("n,dtype", [(1, BF), (40, HF), (3, F32)])
def test_sequences_that_share_their_first_blocks(ctx, n, dtype):
    """One prompt's blocks in the tables of three sequences that go on by themselves."""
    B, Hq, H, cap, shared = 3, 8, 2, 448, 256
    lens = [300, 256 + n, 448]
    nblk = cap // 64
    table = torch.zeros(B, H, nblk, dtype=torch.int32, device=DEV)
    own = torch.arange(B * H * nblk, dtype=torch.int32, device=DEV).view(B, H, nblk)
    table[:] = own
    table[:, :, :shared // 64] = own[:1, :, :shared // 64]
    cache = tq.PagedCache(ctx, B, H, cap, B * H * nblk, table, device=DEV)
    k, v = queries(1, B, H, cap, BF), queries(2, B, H, cap, BF)
    tq.tq_q8_append(ctx.handle, cache, k[:, :, :shared], v[:, :, :shared], ints([0] * B), new_lens=ints([shared, 0, 0]))
    tq.tq_q8_append(ctx.handle, cache, k[:, :, shared:], v[:, :, shared:], ints([shared] * B), new_lens=ints([x - shared for x in lens]))
    kv, vv = (np64(t) for t in tq.tq_dequantize(ctx.handle, cache, 0, cap))
    q = queries(3, B, Hq, n, dtype)
    w = torch.empty(B, H, cap, device=DEV)
    got = tq.tq_q8_attention(ctx.handle, cache, q, ints(lens), cap, weights=w)
    check(np64(got), np64(q), kv, vv, lens, [n] * B, dtype=dtype, out_dtype=dtype, weights=np64(w))


def test_a_general_step_as_a_graph(ctx):
    """tq_decode_step on an 8-bit cache, captured and replayed while its lengths and inputs change."""
    B, Hq, H, cap = 3, 8, 2, 320
    a, b = (make(ctx, B, H, cap, [255, 64, 0], seed=9, poison=False)[0] for _ in range(2))
    q, kn, vn = queries(5, B, Hq, 1, BF)[:, :, 0].contiguous(), queries(6, B, H, 1, BF), queries(7, B, H, 1, BF)
    lens = ints([255, 64, 0])
    ws = torch.empty(tq.tq_workspace_size(ctx.handle, B, Hq, H, cap), dtype=torch.uint8, device=DEV)
    out, ref = torch.empty(B, Hq, 128, device=DEV), torch.empty(B, Hq, 128, device=DEV)
    tq.tq_decode_step(ctx.handle, make(ctx, B, H, cap, [1, 1, 1], seed=1)[0], q, kn, vn, ints([1, 1, 1]), cap, workspace=ws, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_decode_step(ctx.handle, a, q, kn, vn, lens, cap, workspace=ws, out=out)
    for i in range(5):
        q.copy_(queries(20 + i, B, Hq, 1, BF)[:, :, 0])
        kn.copy_(queries(30 + i, B, H, 1, BF, size=1.0 + i))
        g.replay()
        tq.tq_decode_step(ctx.handle, b, q, kn, vn, lens, cap, out=ref)
        assert torch.equal(out, ref)
        lens += 1
    for name in a.tensors:
        assert torch.equal(a.tensors[name], b.tensors[name])


def test_rotary_on_a_context_of_another_scheme():
    other, own = tq.Context(128, 4, "KQV", 1), tq.Context(128, 8, "Q8", 1)
    x, pos = queries(1, 2, 3, 40, BF), torch.arange(80, dtype=torch.int32, device=DEV).view(2, 40)
    for c in (other, own):
        tq.tq_set_rope(c.handle, 64, True, base=500000.0)
    assert torch.equal(tq.tq_rotary(other.handle, x, pos), tq.tq_rotary(own.handle, x, pos))
    other.close()
    own.close()
