"""Workloads of the 8-bit cache path: rotary positions, the quantising append, attention over the
cache (single tokens and prompts; capped scores, distance bias, key ranges; accumulated attention
weight) and eviction by that weight -- each in a plain torch form and as the library's calls.

Layout of the 8-bit cache, as include/tq.h states it: blocks of 64 token slots, [batch][heads_kv]
[ceil(capacity / 64)] of them, 16384 bytes each: an 8192-byte key plane, then the value plane. A
plane holds its 64 tokens in groups of 8; a group is eight 16-byte columns of the head dimension,
each with its 8 tokens' 16 bytes one after the other. Codes are float8 e4m3; each plane of a block
has one power-of-two scale (float32 [block])."""

import math
import random

import numpy as np
import torch

own = False  # True: run() makes the library's calls

D = 128      # head dimension
BLK = 64     # token slots of a block
E_MIN = -100  # smallest block exponent

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # the query rotation of one decode step of a batch: latency
        dict(name="rotary step b16 h32", op="rotary", dtype="bf16", batch=16, heads=32, n=1, dim=128, interleaved=False,
             base=10000.0, factor=1.0, start=8191, token_major=False, salt=1),
        # a long prompt's queries, projection order [token][head], half of the head, scaled for a longer context
        dict(name="rotary prompt 16k part", op="rotary", dtype="bf16", batch=1, heads=32, n=16384, dim=64, interleaved=True,
             base=500000.0, factor=8.0, start=100001, token_major=True, salt=2),
        # one decode step's new tokens of a ragged batch, rotated on the way into the cache
        dict(name="append step b16 h8", op="append", dtype="bf16", batch=16, heads_kv=8, n=1, longest=2047, ragged=True, rope=True,
             token_major=False, salt=3),
        # four prompts written in bulk from the projection's order
        dict(name="append prompts 4x16384", op="append", dtype="bf16", batch=4, heads_kv=8, n=16384, longest=0, ragged=False,
             rope=True, token_major=True, salt=4),
        # one short sequence, grouped heads, the attention weight accumulated for a later eviction: latency
        dict(name="decode 1000 weights", op="attend", dtype="bf16", batch=1, heads_q=32, heads_kv=8, n_q=1, longest=1000,
             ragged=False, softcap=0.0, bias=False, mask="causal", weights=True, paged=False, salt=5),
        # a serving batch with one query head per KV head: the cache's bytes
        dict(name="decode b16 h32 8192", op="attend", dtype="bf16", batch=16, heads_q=32, heads_kv=32, n_q=1, longest=8192,
             ragged=False, softcap=0.0, bias=False, mask="causal", weights=False, paged=False, salt=6),
        # one long context, grouped heads, capped scores, blocks scattered in a pool
        dict(name="decode 131072 capped paged", op="attend", dtype="bf16", batch=1, heads_q=32, heads_kv=8, n_q=1, longest=131072,
             ragged=False, softcap=30.0, bias=False, mask="causal", weights=False, paged=True, salt=7),
        # three drafted tokens a sequence, ragged lengths, float32, distance bias, weight accumulated
        dict(name="draft fp32 bias weights", op="attend", dtype="fp32", batch=4, heads_q=16, heads_kv=8, n_q=3, longest=16383,
             ragged=True, softcap=0.0, bias=True, mask="causal", weights=True, paged=False, salt=8),
        # the last 2048 tokens of an 8192-token prompt
        dict(name="prompt 2048 of 8192", op="attend", dtype="bf16", batch=1, heads_q=32, heads_kv=8, n_q=2048, longest=8192,
             ragged=False, softcap=0.0, bias=False, mask="causal", weights=False, paged=False, token_major=True, salt=9),
        # packed documents behind a shared prefix, capped scores, ragged
        dict(name="prompts documents capped", op="attend", dtype="fp16", batch=4, heads_q=16, heads_kv=4, n_q=1001, longest=4001,
             ragged=True, softcap=50.0, bias=False, mask="documents", weights=False, paged=False, token_major=True, salt=10),
        # one long context cut to a budget
        dict(name="evict 131072 to 4096", op="evict", batch=1, heads_kv=8, longest=131072, ragged=False, keep=4096, sink=4, recent=128,
             salt=11),
        # a ragged batch cut to half its longest
        dict(name="evict b16 8192 to 4000", op="evict", batch=16, heads_kv=8, longest=8192, ragged=True, keep=4000, sink=16, recent=512,
             salt=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    salt = rng.randrange(1, 1 << 30)
    op = rng.choice(["rotary", "append", "attend", "attend", "attend", "evict"])
    dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "rotary":
        heads = rng.choice([1, 3, 8, 32, 40])
        batch = rng.choice([1, 2, 5, 16])
        n = _log(rng, 1, max(2, 262144 // (heads * batch)))
        return dict(op=op, dtype=dt, batch=batch, heads=heads, n=n, dim=rng.choice([32, 64, 72, 128]), interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 32.0]), start=_log(rng, 1, 1000000),
                    token_major=rng.random() < 0.5, salt=salt)
    if op == "append":
        batch, heads = rng.choice([1, 3, 16, 33]), rng.choice([1, 4, 8, 32])
        n = _log(rng, 1, max(2, 400000 // (heads * batch)))
        return dict(op=op, dtype=dt, batch=batch, heads_kv=heads, n=n, longest=_log(rng, 1, 2000) - 1, ragged=rng.random() < 0.7,
                    rope=rng.random() < 0.5, token_major=rng.random() < 0.5, salt=salt)
    if op == "evict":
        batch, heads = rng.choice([1, 4, 16]), rng.choice([1, 8, 20])
        longest = _log(rng, 200, max(400, 1048576 // (heads * batch)))
        keep = max(40, int(longest * rng.uniform(0.03, 0.9)))
        return dict(op=op, batch=batch, heads_kv=heads, longest=longest, ragged=rng.random() < 0.6, keep=keep, sink=rng.choice([0, 1, 4, 13]),
                    recent=rng.randrange(0, keep - 16), salt=salt)
    heads_kv, group = rng.choice([1, 4, 8, 32]), rng.choice([1, 2, 3, 4, 7, 8, 16])
    mask = rng.choice(["causal", "causal", "window", "documents"])
    if rng.random() < 0.6:  # single tokens and drafts
        batch, n_q = rng.choice([1, 2, 7, 16, 40]), rng.choice([1, 1, 1, 2, 5])
        longest = max(n_q, _log(rng, 1, max(64, 2097152 // (batch * heads_kv * max(1, group * n_q // 4)))))
    else:  # prompts
        batch = rng.choice([1, 2, 4])
        n_q = _log(rng, 6, max(32, 65536 // (batch * heads_kv * group)))
        longest = n_q + _log(rng, 1, 6000) - 1
    return dict(op=op, dtype=dt, batch=batch, heads_q=heads_kv * group, heads_kv=heads_kv, n_q=n_q, longest=longest,
                ragged=rng.random() < 0.5, softcap=rng.choice([0.0, 0.0, 20.0]), bias=rng.random() < 0.3, mask=mask,
                weights=rng.random() < 0.25, paged=rng.random() < 0.3, token_major=rng.random() < 0.5, salt=salt)


def _lens(c, least):
    """The sequences' lengths: all `longest`, or spread between `least` and it."""
    if not c["ragged"]:
        return [c["longest"]] * c["batch"]
    r = random.Random(c["salt"])
    return [c["longest"]] + [r.randint(min(least, c["longest"]), c["longest"]) for _ in range(c["batch"] - 1)]


def _new_lens(c):
    """The query tokens of each sequence (ragged batches: some bring fewer)."""
    if not c["ragged"] or c["n_q"] == 1:
        return [c["n_q"]] * c["batch"]
    r = random.Random(c["salt"] + 1)
    return [c["n_q"]] + [r.randint(1, c["n_q"]) for _ in range(c["batch"] - 1)]


def _ranges(c):
    """Key ranges [begin, end) of every query token, as lists [batch][n_q]; rows past a sequence's query tokens are (0, 0)."""
    r = random.Random(c["salt"] + 2)
    begin, end = [], []
    for n, m in zip(_lens(c, c["n_q"]), _new_lens(c)):
        at = np.arange(n - m, n)
        if c["mask"] == "window":  # the last `w` tokens
            w = r.randint(1, max(1, n))
            lo, hi = np.maximum(0, at + 1 - w), at + 1
        elif c["mask"] == "documents":  # documents of a few hundred tokens; the first tokens see a prefix in both directions
            cuts = np.array(sorted({0} | {r.randrange(n) for _ in range(n // 300)}))
            lo = cuts[np.searchsorted(cuts, at, side="right") - 1]
            prefix = n - m + r.randint(0, max(1, m // 4))
            hi = np.maximum(at + 1, np.minimum(prefix, n))
        else:
            lo, hi = 0 * at, at + 1
        pad = np.zeros(c["n_q"] - m, dtype=np.int64)
        begin.append(np.concatenate([lo, pad]))
        end.append(np.concatenate([hi, pad]))
    return np.stack(begin), np.stack(end)


def _blocks(n):
    return (n + BLK - 1) // BLK


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _vectors(g, c, batch, heads, n, scales=True):
    """[batch][heads][n][D] activations with channels of unequal size, in the case's type and order of dimensions."""
    x = _randn(g, batch, heads, n, D)
    if scales:
        x = x * torch.exp(0.5 * _randn(g, 1, heads, 1, D))
    x = x.to(_DT[c["dtype"]])
    if c.get("token_major"):  # [batch][token][head][D] storage
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    return x


def _rope_case(c):
    """(dim, interleaved, base, factor, original length, low, high, output factor) of the case's rotation."""
    if c["op"] == "append":
        return dict(dim=D, interleaved=False, base=10000.0, factor=1.0, original=8192, low=1.0, high=4.0, gain=1.0)
    return dict(dim=c["dim"], interleaved=c["interleaved"], base=c["base"], factor=c["factor"], original=8192, low=1.0, high=4.0,
                gain=1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0)


def _fill(g, batch, heads, nblk):
    """Codes and scales of a cache's blocks: (records uint8 [blocks][16384], key scales, value scales [blocks])."""
    k = _randn(g, batch * heads * nblk, BLK, D) * torch.exp(0.5 * _randn(g, 1, 1, D))
    v = _randn(g, batch * heads * nblk, BLK, D)
    kc, ks = _quantise(k)
    vc, vs = _quantise(v)
    return torch.cat([_to_plane(kc), _to_plane(vc)], 1), ks, vs


def _library(c):
    """The library's context, with the case's rotation set."""
    from quantised_kv_cache_gb300 import tq
    ctx = tq.Context(D, 8, "Q8", 42)
    if c["op"] in ("rotary", "append"):
        r = _rope_case(c)
        tq.tq_set_rope(ctx.handle, r["dim"], interleaved=r["interleaved"], base=r["base"], factor=r["factor"],
                       original_len=r["original"], low=r["low"], high=r["high"], gain=r["gain"])
    return tq, ctx


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + c["salt"])
    s = {"case": c}
    ints = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    if c["op"] == "rotary":
        s["x"] = _vectors(g, c, c["batch"], c["heads"], c["n"])
        s["pos"] = ints(c["start"] + np.arange(c["n"]) + 17 * np.arange(c["batch"])[:, None])
        if own:
            s["tq"], s["ctx"] = _library(c)
        return s
    if c["op"] == "append":
        lens = _lens(c, 0)
        nblk = _blocks(max(lens) + c["n"])
        s["k"] = _vectors(g, c, c["batch"], c["heads_kv"], c["n"])
        s["v"] = _vectors(g, c, c["batch"], c["heads_kv"], c["n"])
        s["lens"], s["nblk"] = ints(lens), nblk
        s["reach"] = max(_blocks(n % BLK + c["n"]) for n in lens)  # blocks a sequence's new tokens lie in, at most
        s["records"], s["ks"], s["vs"] = _fill(g, c["batch"], c["heads_kv"], nblk)
    elif c["op"] == "evict":
        lens = _lens(c, 0)
        nblk = _blocks(max(max(lens), 1))
        s["lens"], s["nblk"] = ints(lens), nblk
        s["records"], s["ks"], s["vs"] = _fill(g, c["batch"], c["heads_kv"], nblk)
        # a few heavy tokens, many light ones; one in sixteen has no weight, so that there are ties
        w = torch.exp(2.0 * _randn(g, c["batch"], c["heads_kv"], nblk * BLK))
        s["w"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 1 / 16, torch.zeros_like(w), w)
        s["pos"] = torch.arange(nblk * BLK, dtype=torch.int32, device="cuda").expand(w.shape).contiguous() * 2
    else:
        lens = _lens(c, c["n_q"])
        nblk = _blocks(max(lens))
        s["lens"], s["new"], s["nblk"] = ints(lens), ints(_new_lens(c)), nblk
        begin, end = _ranges(c)
        s["begin"], s["end"] = ints(begin), ints(end)
        s["q"] = _vectors(g, c, c["batch"], c["heads_q"], c["n_q"], scales=False)
        s["records"], s["ks"], s["vs"] = _fill(g, c["batch"], c["heads_kv"], nblk)
        s["table"] = None
        if c["paged"]:
            s["table"] = torch.randperm(s["ks"].numel(), generator=g, device="cuda").to(torch.int32).view(c["batch"], c["heads_kv"], nblk)
        if c["bias"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["heads_q"] + 1, device="cuda", dtype=torch.float32) / c["heads_q"])
        if c["weights"]:
            s["acc"] = _randn(g, c["batch"], c["heads_kv"], nblk * BLK).abs()
    if own:  # the same blocks in the library's cache
        tq, ctx = s["tq"], s["ctx"] = _library(c)
        if c["op"] == "attend" and c["paged"]:
            cache = tq.PagedCache(ctx, c["batch"], c["heads_kv"], nblk * BLK, s["ks"].numel(), s["table"])
        else:
            cache = tq.Cache(ctx, c["batch"], c["heads_kv"], nblk * BLK)
        cache.tensors["records"].copy_(s["records"].view(-1))
        cache.tensors["k_stats"].view(torch.float32).copy_(s["ks"])
        cache.tensors["v_stats"].view(torch.float32).copy_(s["vs"])
        s["cache"] = cache
        if c["op"] == "evict":
            s["dst"] = tq.Cache(ctx, c["batch"], c["heads_kv"], _blocks(c["keep"]) * BLK)
        if c["op"] == "attend":
            s["ws"] = torch.empty(tq.tq_q8_attention_workspace(ctx.handle, c["batch"], c["heads_q"], c["heads_kv"], c["n_q"], nblk * BLK,
                                                                 weights=c["weights"]),
                                  dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------

def _pow2(e):
    """2^e of whole numbers e in [-126, 127], exactly (the exponent field of a float32)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_of(amax):
    """2^e, e the least integer >= E_MIN with amax <= 448 * 2^e (0.875 <= m < 1 in amax = m 2^x: m 2^x <= 0.875 * 2^9 * 2^e)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(min=E_MIN)
    return _pow2(e)


def _round8(x):
    """x rounded to e4m3 (to nearest, ties to even), |x| <= 448: steps of 2^(e - 3), of 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = _pow2(torch.clamp(e - 1, min=-6) - 3)
    return (torch.round(x / step) * step).to(torch.float8_e4m3fn)


def _quantise(x):
    """[blocks][BLK][D] -> codes, scales."""
    scale = _scale_of(x.abs().amax((1, 2)))
    return _round8(x / scale[:, None, None]), scale


def _to_plane(codes):
    """[blocks][BLK][D] float8 -> [blocks][8192] bytes in the cache's order."""
    n = codes.shape[0]
    return codes.view(torch.uint8).view(n, BLK // 8, 8, D // 16, 16).transpose(2, 3).reshape(n, BLK * D)


def _from_plane(plane):
    """[blocks][8192] bytes -> [blocks][BLK][D] float32."""
    n = plane.shape[0]
    return plane.view(n, BLK // 8, D // 16, 8, 16).transpose(2, 3).reshape(n, BLK, D).view(torch.float8_e4m3fn).float()


def _inverse_lengths(r, device):
    """Radians a position of each pair, in 64 bits: base^(-2i/dim); with a factor, divided by it where the pair turns fewer than `low`
    times in the original length, kept where it turns more than `high` times, blended between."""
    f = r["base"] ** (-torch.arange(0, r["dim"], 2, dtype=torch.float64, device=device) / r["dim"])
    if r["factor"] == 1.0:
        return f
    turns = r["original"] * f / (2 * math.pi)
    keep = ((turns - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
    return f * keep + f / r["factor"] * (1 - keep)


def _rotated(x, pos, r):
    """x [B][H][n][D] at positions pos [B][n]: angles in 64 bits, the rotation in 32, rounded to x's type."""
    angle = pos.double()[:, None, :, None] * _inverse_lengths(r, x.device)
    cos, sin = (angle.cos() * r["gain"]).float(), (angle.sin() * r["gain"]).float()
    y, dim = x.float(), r["dim"]
    if r["interleaved"]:
        a, b = y[..., 0:dim:2], y[..., 1:dim:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :dim // 2], y[..., dim // 2:dim]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., dim:]], -1).to(x.dtype)


def _append_plane(plane, scale, x, lens, reach, nblk):
    """New tokens x [B][H][n][D] into the blocks they fall in: `plane` [B*H*nblk][8192], `scale` [B*H*nblk], in place."""
    B, H, n, _ = x.shape
    dev = x.device
    first = lens.long() // BLK                                                       # [B]
    blk = first[:, None] + torch.arange(reach, device=dev)                           # [B][reach]
    there = blk * BLK < lens.long()[:, None] + n                                     # blocks the call writes
    row = (torch.arange(B * H, device=dev).view(B, H, 1) * nblk + blk.clamp(max=nblk - 1)[:, None, :])[there[:, None, :].expand(B, H, reach)]
    slot = blk[:, :, None] * BLK + torch.arange(BLK, device=dev) - lens.long()[:, None, None]  # new token of each slot
    new = ((slot >= 0) & (slot < n))
    old = slot < 0
    at = slot.clamp(0, n - 1).view(B, 1, reach * BLK, 1).expand(B, H, reach * BLK, D)
    pick = there[:, None, :].expand(B, H, reach)
    y = torch.gather(x, 2, at).view(B, H, reach, BLK, D)[pick].float()               # [rows][BLK][D]
    new = new[:, None].expand(B, H, reach, BLK)[pick][..., None]
    old = old[:, None].expand(B, H, reach, BLK)[pick][..., None]
    codes, was = _from_plane(plane[row]), scale[row]
    need = _scale_of(torch.where(new, y, torch.zeros_like(y)).abs().amax((1, 2)))
    now = torch.where(old.any(1).squeeze(-1), torch.maximum(need, was), need)
    kept = _round8(codes * (was / now)[:, None, None])
    put = _round8(torch.where(new, y, torch.zeros_like(y)) / now[:, None, None])
    stay = codes.to(torch.float8_e4m3fn)                                             # slots past the new tokens
    out = torch.where(new, put.float(), torch.where(old, kept.float(), stay.float())).to(torch.float8_e4m3fn)
    plane[row] = _to_plane(out)
    scale[row] = now


def _cache_values(s, c):
    """(keys, values) [B][H][slots][D] float32 that a state's blocks stand for."""
    pick = slice(None) if s.get("table") is None else s["table"].view(-1).long()
    rec = s["records"][pick]
    shape = (c["batch"], c["heads_kv"], s["nblk"] * BLK, D)
    half = BLK * D
    return ((_from_plane(rec[:, :half]) * s["ks"][pick][:, None, None]).view(shape),
            (_from_plane(rec[:, half:]) * s["vs"][pick][:, None, None]).view(shape))


def _attend_plain(s, c):
    k, v = _cache_values(s, c)
    B, Hq, Hkv, n, N = c["batch"], c["heads_q"], c["heads_kv"], c["n_q"], s["nblk"] * BLK
    q = s["q"].float().reshape(B, Hkv, (Hq // Hkv) * n, D)
    t = (q @ k.transpose(-1, -2)).view(B, Hq, n, N) * (1.0 / math.sqrt(D))
    if c["softcap"]:
        t = c["softcap"] * torch.tanh(t / c["softcap"])
    slot = torch.arange(N, device=q.device)
    if c["bias"]:
        at = s["lens"][:, None] - s["new"][:, None] + torch.arange(n, device=q.device)          # the queries' own slots
        t = t - s["slopes"][:, None, None] * (at[:, :, None] - slot).abs()[:, None].float()
    seen = (slot >= s["begin"][..., None]) & (slot < s["end"][..., None])                       # [B][n][N]
    t = torch.where(seen[:, None], t, torch.full_like(t, float("-inf")))
    top = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    out = (p.view(B, Hkv, (Hq // Hkv) * n, N) @ v).view(B, Hq, n, D).to(s["q"].dtype)
    if not c["weights"]:
        return {"out": out}
    return {"out": out, "weights": s["acc"] + p.view(B, Hkv, -1, N).sum(2)}


def _evict_plain(s, c):
    B, H, N, keep = c["batch"], c["heads_kv"], s["nblk"] * BLK, c["keep"]
    dev = s["w"].device
    slot = torch.arange(N, device=dev)
    n = s["lens"].long()[:, None, None]
    always = (slot < c["sink"]) | (slot >= n - c["recent"])
    rank = torch.where(always, torch.full_like(s["w"], float("inf")), s["w"])
    rank = torch.where(slot < n, rank, torch.full_like(rank, float("-inf")))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    count = torch.minimum(n, torch.full_like(n, keep))                              # [B][1][1]
    lane = torch.arange(order.shape[-1], device=dev)
    kept = torch.sort(torch.where(lane < count, order, torch.full_like(order, N)), dim=-1).values
    kept = torch.cat([kept, kept.new_full((B, H, keep - kept.shape[-1]), N)], -1)
    lane = torch.arange(keep, device=dev)
    live = lane < count
    at = kept.clamp(max=N - 1)
    zero = lambda t: torch.where(live, t, torch.zeros_like(t))  # noqa: E731
    res = {"kept": torch.where(live, kept, torch.full_like(kept, -1)).int(), "lens": count.view(-1).int(),
           "weights": zero(torch.gather(s["w"], 2, at)), "positions": zero(torch.gather(s["pos"], 2, at))}
    pad = _blocks(keep) * BLK - keep

    def moved(x):
        y = torch.gather(x, 2, at[..., None].expand(B, H, keep, D)) * live.expand(B, H, keep)[..., None]
        y = torch.cat([y, y.new_zeros(B, H, pad, D)], 2).view(-1, BLK, D)
        codes, scale = _quantise(y)
        return _to_plane(codes).view(torch.float8_e4m3fn), scale

    k, v = _cache_values(s, c)
    res["k"], res["k_scale"] = moved(k)
    res["v"], res["v_scale"] = moved(v)
    return res


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_library(s, c)
    if c["op"] == "rotary":
        return {"y": _rotated(s["x"], s["pos"], _rope_case(c))}
    if c["op"] == "append":
        k = s["k"]
        if c["rope"]:
            k = _rotated(k, s["lens"][:, None] + torch.arange(c["n"], device=k.device), _rope_case(c))
        half = BLK * D
        _append_plane(s["records"][:, :half], s["ks"], k, s["lens"], s["reach"], s["nblk"])
        _append_plane(s["records"][:, half:], s["vs"], s["v"], s["lens"], s["reach"], s["nblk"])
        return {"records": s["records"].view(torch.float8_e4m3fn), "ks": s["ks"], "vs": s["vs"]}
    return _attend_plain(s, c) if c["op"] == "attend" else _evict_plain(s, c)


def _run_library(s, c):
    tq, ctx = s["tq"], s["ctx"].handle
    if c["op"] == "rotary":
        return {"y": tq.tq_rotary(ctx, s["x"], s["pos"])}
    cache = s["cache"]
    blocks = lambda ch: (ch.tensors["records"].view(-1, 2 * BLK * D).view(torch.float8_e4m3fn),  # noqa: E731
                         ch.tensors["k_stats"].view(torch.float32), ch.tensors["v_stats"].view(torch.float32))
    if c["op"] == "append":
        tq.tq_q8_append(ctx, cache, s["k"], s["v"], s["lens"], rope=c["rope"])
        rec, ks, vs = blocks(cache)
        return {"records": rec, "ks": ks, "vs": vs}
    if c["op"] == "attend":
        kw = {}
        if c["mask"] != "causal":
            kw.update(key_begin=s["begin"], key_end=s["end"])
        if c["bias"]:
            kw.update(slopes=s["slopes"])
        if c["weights"]:
            kw.update(weights_in=s["acc"], weights=torch.empty_like(s["acc"]))
        # rows past a sequence's query tokens stay as they are: zeros, as in the plain form
        out = (torch.zeros if c["ragged"] and c["n_q"] > 1 else torch.empty)(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        tq.tq_q8_attention(ctx, cache, s["q"], s["lens"], s["nblk"] * BLK, new_lens=s["new"] if c["ragged"] else None,
                           softcap=c["softcap"], workspace=s["ws"], out=out, **kw)
        return {"out": out, "weights": kw["weights"]} if c["weights"] else {"out": out}
    kept, lens, w, pos = tq.tq_q8_evict(ctx, cache, s["dst"], s["lens"], s["w"], c["keep"], sink=c["sink"], recent=c["recent"],
                                        positions=s["pos"])
    rec, ks, vs = blocks(s["dst"])
    return {"kept": kept, "lens": lens, "weights": w[..., :c["keep"]], "positions": pos[..., :c["keep"]],
            "k": rec[:, :BLK * D], "k_scale": ks, "v": rec[:, BLK * D:], "v_scale": vs}


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------

def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[c.get("dtype", "bf16")]
    if c["op"] == "rotary":
        x = c["batch"] * c["heads"] * c["n"] * D
        return {"bytes": 2 * x * size + 4 * c["batch"] * c["n"], "flops": 3 * x * c["dim"] // D}
    if c["op"] == "append":
        x = 2 * c["batch"] * c["heads_kv"] * c["n"] * D
        return {"bytes": x * size + x + 8 * x // (BLK * D), "flops": 3 * x}
    if c["op"] == "evict":
        lens = _lens(c, 0)
        moved = sum(min(n, c["keep"]) for n in lens) * c["heads_kv"]
        return {"bytes": 4 * sum(lens) * c["heads_kv"] + moved * (2 * 2 * D + 4 * 5), "flops": sum(lens) * c["heads_kv"] + 2 * moved * D}
    begin, end = _ranges(c)
    pairs = int((end - begin).clip(0).sum())
    seen = 0
    for lo, hi in zip(begin, end):  # slots that some query of the sequence sees
        mark = np.zeros(c["longest"] + 1, dtype=np.int64)
        live = hi > lo
        np.add.at(mark, lo[live], 1)
        np.add.at(mark, hi[live], -1)
        seen += int((np.cumsum(mark) > 0).sum())
    rows = sum(_new_lens(c)) * c["heads_q"]
    return {"bytes": seen * c["heads_kv"] * 2 * D + 2 * rows * D * size + (8 * c["batch"] * c["heads_kv"] * _blocks(c["longest"]) * BLK if c["weights"] else 0),
            "flops": 4 * D * pairs * c["heads_q"]}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------

_GRID = None


def _grid64():
    """The 127 non-negative e4m3 numbers, ascending, in 64 bits."""
    global _GRID
    if _GRID is None:
        _GRID = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8) if (e, m) != (15, 7)])
    return _GRID


def _code64(x):
    """float64 array -> the nearest e4m3 number (ties to the even one of the two codes)."""
    g = torch.as_tensor(_grid64(), device=x.device)
    a = x.abs().contiguous()
    hi = torch.searchsorted(g, a).clamp(max=len(g) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = g[hi] - a, a - g[lo]
    take = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.sign(x) * g[take]


def _two64(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exponent64(amax):
    """The least e >= E_MIN with amax <= 448 * 2^e."""
    e = torch.ceil(torch.log2((amax / 448.0).clamp(min=2.0 ** -200)))
    e = torch.where(448.0 * _two64(e - 1) >= amax, e - 1, e)
    return torch.where(448.0 * _two64(e) < amax, e + 1, e).clamp(min=E_MIN)


def _unpack64(records, which):
    n = records.shape[0]
    plane = records[:, which * BLK * D:(which + 1) * BLK * D].reshape(n, BLK // 8, D // 16, 8, 16)
    return plane.permute(0, 1, 3, 2, 4).reshape(n, BLK, D).contiguous().view(torch.float8_e4m3fn).double()


def _pack64(values):
    n = values.shape[0]
    return values.view(n, BLK // 8, 8, D // 16, 16).permute(0, 1, 3, 2, 4).reshape(n, BLK * D)


def _rotate64(x, pos, r):
    i = torch.arange(r["dim"] // 2, dtype=torch.float64, device=x.device)
    freq = torch.pow(torch.tensor(r["base"], dtype=torch.float64, device=x.device), -2.0 * i / r["dim"])
    if r["factor"] != 1.0:
        share = (r["original"] / (2 * math.pi / freq) - r["low"]) / (r["high"] - r["low"])
        share = torch.minimum(torch.maximum(share, torch.zeros_like(share)), torch.ones_like(share))
        freq = (1 - share) * freq / r["factor"] + share * freq
    z = torch.polar(torch.full_like(freq, r["gain"]).expand(pos.shape + freq.shape), pos[..., None].double() * freq)[:, None]
    x = x.double()
    first, second = (slice(0, r["dim"], 2), slice(1, r["dim"], 2)) if r["interleaved"] else (slice(0, r["dim"] // 2), slice(r["dim"] // 2, r["dim"]))
    y = torch.complex(x[..., first], x[..., second]) * z
    out = x.clone()
    out[..., first], out[..., second] = y.real, y.imag
    return out


def _numpy(d):
    return {k: v.cpu().numpy() for k, v in d.items()}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "rotary":
        return _numpy({"y": _rotate64(s["x"], s["pos"], _rope_case(c))})
    nblk, H, B = s["nblk"], c["heads_kv"], c["batch"]
    if c["op"] == "append":
        n = c["n"]
        at = s["lens"].long()[:, None] + torch.arange(n, device="cuda")
        # the new keys are rounded to their own type before they are quantised
        k = _rotate64(s["k"], at, _rope_case(c)).to(s["k"].dtype) if c["rope"] else s["k"]
        parts, scales = [], []
        for which, (x, scale) in enumerate(((k, s["ks"]), (s["v"], s["vs"]))):
            x = x.double()
            codes, e = _unpack64(s["records"], which).view(B, H, nblk, BLK, D), torch.round(torch.log2(scale.double())).view(B, H, nblk)
            for b in range(B):
                n0 = int(s["lens"][b])
                j0, j1 = n0 // BLK, _blocks(n0 + n)
                wide = torch.zeros(H, (j1 - j0) * BLK, D, dtype=torch.float64, device="cuda")
                wide[:, n0 - j0 * BLK:n0 - j0 * BLK + n] = x[b]
                need = _exponent64(wide.view(H, j1 - j0, BLK * D).abs().amax(-1))
                if n0 % BLK:
                    need[:, 0] = torch.maximum(need[:, 0], e[b, :, j0])
                    codes[b, :, j0, :n0 % BLK] = _code64(codes[b, :, j0, :n0 % BLK] * _two64(e[b, :, j0] - need[:, 0])[:, None, None])
                put = _code64(wide.view(H, j1 - j0, BLK, D) * _two64(-need)[..., None, None]).view(H, -1, D)
                flat = codes[b].view(H, nblk * BLK, D)
                flat[:, n0:n0 + n] = put[:, n0 - j0 * BLK:n0 - j0 * BLK + n]
                e[b, :, j0:j1] = need
            parts.append(_pack64(codes.view(-1, BLK, D)))
            scales.append(_two64(e).view(-1))
        return _numpy({"records": torch.cat(parts, 1), "ks": scales[0], "vs": scales[1]})
    values = []
    for which, scale in enumerate((s["ks"], s["vs"])):
        values.append((_unpack64(s["records"], which), scale.double()))
    if c["op"] == "evict":
        N, keep = nblk * BLK, c["keep"]
        res = {"kept": -torch.ones(B, H, keep, dtype=torch.int32), "lens": torch.zeros(B, dtype=torch.int32),
               "weights": torch.zeros(B, H, keep, dtype=torch.float64), "positions": torch.zeros(B, H, keep, dtype=torch.int32)}
        w, pos = s["w"].cpu().double(), s["pos"].cpu()
        for b in range(B):
            n = int(s["lens"][b])
            m = min(n, keep)
            res["lens"][b] = m
            for h in range(H):
                if n <= keep:
                    took = np.arange(n)
                else:
                    middle = np.arange(c["sink"], n - c["recent"])
                    best = middle[np.lexsort((middle, -w[b, h, middle].numpy()))][:keep - c["sink"] - c["recent"]]
                    took = np.concatenate([np.arange(c["sink"]), np.sort(best), np.arange(n - c["recent"], n)])
                took = torch.as_tensor(took)
                res["kept"][b, h, :m] = took.int()
                res["weights"][b, h, :m], res["positions"][b, h, :m] = w[b, h, took], pos[b, h, took]
        slots = _blocks(keep) * BLK
        at = torch.cat([res["kept"].long(), torch.full((B, H, slots - keep), -1)], -1).cuda()
        for name, (code, scale) in zip("kv", values):
            full = (code * scale[:, None, None]).view(B, H, N, D)
            y = torch.gather(full, 2, at.clamp(min=0)[..., None].expand(B, H, slots, D)) * (at >= 0)[..., None]
            y = y.view(-1, BLK, D)
            e = _exponent64(y.abs().amax((1, 2)))
            res[name], res[name + "_scale"] = _pack64(_code64(y * _two64(-e)[:, None, None])), _two64(e)
        return _numpy(res)
    if 4 * D * float(B) * c["heads_q"] * c["n_q"] * nblk * BLK > 4e12:
        return None
    G, N = c["heads_q"] // H, nblk * BLK
    order = torch.arange(values[0][1].numel(), device="cuda") if s["table"] is None else s["table"].view(-1).long()
    order = order.view(B, H, nblk)
    out = torch.zeros(B, c["heads_q"], c["n_q"], D, dtype=torch.float64, device="cuda")
    acc = s["acc"].double().clone() if c["weights"] else None
    slot = torch.arange(N, device="cuda")
    for b in range(B):
        seen = (slot >= s["begin"][b, :, None]) & (slot < s["end"][b, :, None])
        home = int(s["lens"][b] - s["new"][b]) + torch.arange(c["n_q"], device="cuda")
        for h in range(H):
            k, v = ((code[order[b, h]] * scale[order[b, h]][:, None, None]).view(N, D) for code, scale in values)
            for j in range(h * G, (h + 1) * G):
                t = (s["q"][b, j].double() @ k.T) / math.sqrt(D)
                if c["softcap"]:
                    t = c["softcap"] * torch.tanh(t / c["softcap"])
                if c["bias"]:
                    t = t - s["slopes"][j].double() * (home[:, None] - slot).abs()
                t = t.masked_fill(~seen, float("-inf"))
                p = torch.nan_to_num(torch.softmax(t, -1), nan=0.0)
                out[b, j] = p @ v
                if acc is not None:
                    acc[b, h] += p.sum(0)
    return _numpy({"out": out, "weights": acc} if c["weights"] else {"out": out})
