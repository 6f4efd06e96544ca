"""A bound on the roundings of the 8-bit cache's attention kernels, per row, from the row's own inputs.

The products' sums are off by at most 130 U of the sum of their magnitudes (fp32, any order, three scalings). A query enters as 8-bit
terms with its row's largest coordinate near the top: 16-bit coordinates of at least 2^-9 of the largest exactly, smaller ones within
2^-20 of it (many rows in bf16: 2^-17; 32-bit results 2^-31), float32 ones within 2^-22 of themselves and 2^-31 of the largest (32-bit results
only; else as 16-bit ones, after their own rounding to the terms' 2^-11). Capping, bias and the exponent add a few U of what they handle (a cap by the short tanh of many rows
2^-21 of the cap); a probability's relative error is twice the largest score error (its own and the sum's) and 2^-20 for the two exponentials.
Probabilities enter the value sums as terms: 2^-11 of each and 2^-21 of the largest (few rows 16-bit results), 2^-11 and 2^-17 (many rows,
fp16), 2^-8 and 2^-14 (many, bf16), 2^-22 and 2^-32 (32-bit results), never more than itself. Sums over tiles of 128 add U each, the join of two parts
2^-20 of either; the result is rounded to its type."""

import numpy as np
import torch

from oracle import q8_blocks as ob

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def assert_rows(got, q, k, v, seen, *, dtype, out_dtype, many, scale=None, softcap=0.0, slope=0.0, distance=None, lse=None, joined=False):
    """got, q [m][128], k, v [N][128] float64, seen [m][N]; `many`: more than 16 rows to a unit (any of the parts)."""
    m, N = seen.shape
    if m == 0:
        return 0.0
    distance = np.zeros(seen.shape) if distance is None else distance
    sc = 1 / np.sqrt(128.0) if scale is None else scale
    wide = out_dtype == F32
    many = many and not wide
    want, p, wl = ob.attend(q, k, v, seen, scale=sc, softcap=softcap, slope=slope, distance=distance)
    big = np.abs(q).max(-1, keepdims=True)
    if dtype == F32:
        dq = 2.0 ** -22 * np.abs(q) + 2.0 ** -31 * big
    else:
        dq = np.where(np.abs(q) < 2.0 ** -9 * big, (2.0 ** -31 if wide else 2.0 ** -17 if many and dtype == BF else 2.0 ** -20) * big, 0.0)
    e = sc * (dq @ np.abs(k).T) + 130 * U * sc * (np.abs(q) @ np.abs(k).T)
    e = e + 8 * U * (softcap * (2 if many else 1) + np.abs(slope * distance) + sc * np.abs(q @ k.T))
    e = np.where(p > 0, e, 0).max(-1, keepdims=True, initial=0.0)
    rel = 2 * e + 2.0 ** -20 + (2.0 ** -19 if joined else 0.0)
    term, floor = (2.0 ** -22, 2.0 ** -32) if wide else (2.0 ** -8, 2.0 ** -14) if many and dtype == BF else (2.0 ** -11, 2.0 ** -17 if many else 2.0 ** -21)
    sums = 2 * (140 + N / 128) * U
    tol = (rel + sums) * (p @ np.abs(v))
    tol += 2 * (np.minimum(p, term * p + floor * p.max(-1, keepdims=True, initial=0.0)) @ np.abs(v))
    tol += np.abs(want) * torch.finfo(out_dtype).eps / 2 * 1.01 + (1e-30 if wide or out_dtype == BF else 2.0 ** -25)
    err = np.abs(got - want)
    assert np.all(err <= tol), (err / tol).max()
    if lse is not None:
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(lse), empty)
        wl, e = wl[~empty], e[~empty, 0]
        assert np.all(np.abs(lse[~empty] - wl) <= e + 2.0 ** -19 + sums + 4 * U * np.abs(wl))
    return (err / tol).max()
