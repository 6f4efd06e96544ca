"""Bounds and choice of blocks of the 8-bit cache, attention over listed blocks and behind a shared prefix, restated in
fp64 and whole numbers (numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``). The rules are those of include/tq.h: "Bounds of each block's keys",
tq_q8_pick, tq_q8_sparse_attention, tq_q8_shared_attention.
"""

import numpy as np

BLOCK = 64


def bounds(codes):
    """codes [tokens][128] (values of e4m3 numbers) of one block -> (lo, hi) int [128], in steps of 4 codes."""
    return np.floor(codes.min(0) / 4.0).astype(int), np.ceil(codes.max(0) / 4.0).astype(int)


def whole_rows(rows):
    """rows [n][128] -> (whole numbers within +-127 on one power of two, which rows count)."""
    rows = np.asarray(rows, dtype=np.float64)
    good = np.isfinite(rows).all(1)
    top = np.abs(rows[good]).max(initial=0.0)
    if top == 0.0:
        return np.zeros(rows.shape, dtype=np.int64), good
    m, x = np.frexp(top)  # top = m 2^x, 1/2 <= m < 1
    w = np.zeros(rows.shape, dtype=np.int64)
    w[good] = np.clip(np.rint(np.ldexp(rows[good], 7 - int(x))), -127, 127).astype(np.int64)  # (rint: ties to even)
    return w, good


def scores(rows, lo, hi, exponents):
    """Exact scores of blocks with bounds lo, hi [blocks][128] and key exponents, as (whole number, exponent) pairs in sortable
    Python form: a list of fractions (int * 2^(e + 200))."""
    w, good = whole_rows(rows)
    if not good.any():
        best = np.zeros(len(lo), dtype=np.int64)
    else:
        w = w[good]
        best = (np.maximum(w, 0) @ hi.astype(np.int64).T + np.minimum(w, 0) @ lo.astype(np.int64).T).max(0)
    return [int(s) * 2 ** (int(e) + 200) for s, e in zip(best, exponents)]


def choose(score, first, last, keep, sink, recent):
    """The blocks of a list that sees blocks first .. last - 1; score[j] of block first + j."""
    if last - first <= keep:
        return list(range(first, last))
    middle = range(first + sink, last - recent)
    best = sorted(middle, key=lambda j: (-score[j - first], j))[:keep - sink - recent]
    return sorted([*range(first, first + sink), *best, *range(last - recent, last)])


def attend(q, k, v, seen, *, scale=None, softcap=0.0, slope=None, distance=None):
    """q [n][128] over k, v [N][128], row i sees the keys with seen[i]. Returns (out, probabilities, natural log of the sum)."""
    t = (q @ k.T) * (1 / np.sqrt(128.0) if scale is None else scale)
    if softcap:
        t = softcap * np.tanh(t / softcap)
    if slope is not None:
        t = t - slope * distance
    t = np.where(seen, t, -np.inf)
    top = t.max(-1, keepdims=True, initial=-np.inf)
    w = np.exp(t - np.where(np.isneginf(top), 0.0, top))
    total = w.sum(-1, keepdims=True)
    p = w / np.where(total > 0, total, 1.0)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, top + np.log(total), -np.inf)[:, 0]
    return p @ np.where(seen.any(0)[:, None], v, 0.0), p, lse
