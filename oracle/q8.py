"""The 8-bit cache and rotary positions, restated in fp64 (numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Storage rule (include/tq.h, "Q8 records"): blocks of 64 tokens; per block and tensor the least whole
e >= -100 with max |x| <= 448 * 2^e over the new finite coordinates, never below the exponent of a block
that already held tokens (whose codes are then rounded to the new scale); code = the e4m3 number
nearest to x * 2^-e, ties to the one with an even code, infinities to +-448, NaN to 0. Finite x are
first cut to +-1.875 * 2^127, so that what a code stands for is finite in float32.
"""

import numpy as np

BLOCK = 64
MIN_EXP = -100
LARGEST = 1.875 * 2.0 ** 127

#: the non-negative e4m3 numbers in code order: (1 + m/8) 2^(e - 7), m/8 2^-6 for e = 0
GRID = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8) if not (e == 15 and m == 7)])


def e4m3(x):
    """The nearest e4m3 numbers of finite or infinite x (float64)."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(GRID, a), 0, len(GRID) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    take = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.copysign(GRID[take], x)


def exponent(amax):
    """The least e >= MIN_EXP with amax <= 448 * 2^e (a Python float)."""
    e = MIN_EXP
    if amax > 0:
        m, x = np.frexp(amax)  # amax = m 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
        e = max(e, int(x) - 9 if m <= 0.875 else int(x) - 8)
    return e


class Model:
    """One tensor (keys or values) of a cache: codes [bh][slots][128] and exponents [bh][blocks]."""

    def __init__(self, heads, capacity):
        blocks = -(-capacity // BLOCK)
        self.codes = np.zeros((heads, blocks * BLOCK, 128))
        self.exp = np.zeros((heads, blocks), dtype=int)

    def append(self, h, at, x):
        """x [n][128] at slots at .. at + n - 1 of sequence-head h, as one call."""
        x = np.asarray(x, dtype=np.float64)
        for j in range(at // BLOCK, -(-(at + len(x)) // BLOCK) if len(x) else 0):
            s0, s1 = max(at, j * BLOCK), min(at + len(x), (j + 1) * BLOCK)
            new = x[s0 - at:s1 - at]
            new = np.where(np.isfinite(new), np.clip(new, -LARGEST, LARGEST), new)
            fin = np.isfinite(new)
            e = exponent(np.max(np.abs(new[fin]), initial=0.0))
            if j * BLOCK < at:
                was = self.exp[h, j]
                e = max(e, was)
                if e > was:
                    old = slice(j * BLOCK, at)
                    self.codes[h, old] = e4m3(self.codes[h, old] * 2.0 ** (was - e))
            self.exp[h, j] = e
            self.codes[h, s0:s1] = e4m3(np.where(np.isnan(new), 0.0, new) * 2.0 ** -e)

    def values(self):
        return self.codes * np.repeat(2.0 ** self.exp, BLOCK, axis=1)[..., None]


def rope_frequencies(dim, base=10000.0, factor=1.0, original_len=0.0, low=0.0, high=0.0):
    f = base ** (-2.0 * np.arange(dim // 2) / dim)
    if factor > 1.0:
        keep = np.zeros_like(f)
        if low or high:
            keep = np.clip((original_len * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = (1 - keep) * f / factor + keep * f
    return f


def rope(x, pos, dim, interleaved=False, gain=1.0, transpose=False, **kw):
    """x [..., n, 128] at positions [..., n]."""
    x = np.array(x, dtype=np.float64)
    ang = np.asarray(pos, dtype=np.float64)[..., None] * rope_frequencies(dim, **kw)
    c, s = gain * np.cos(ang), gain * np.sin(ang) * (-1.0 if transpose else 1.0)
    one, two = (slice(0, dim, 2), slice(1, dim, 2)) if interleaved else (slice(0, dim // 2), slice(dim // 2, dim))
    a, b = x[..., one].copy(), x[..., two].copy()
    x[..., one], x[..., two] = a * c - b * s, b * c + a * s
    return x


def attend(q, k, v, begin, end, *, scale=None, softcap=0.0, slope=None, q_pos=None, k_pos=None):
    """One head: q [n][128] over k, v [N][128], query i sees slots [begin[i], end[i]).
    Returns (out [n][128], probabilities [n][N], natural log of the softmax's sum [n])."""
    n, N = len(q), len(k)
    t = (q @ k.T) * (1 / np.sqrt(128.0) if scale is None else scale)
    if softcap:
        t = softcap * np.tanh(t / softcap)
    if slope is not None:
        t = t - slope * np.abs(np.asarray(q_pos)[:, None].astype(np.float64) - np.asarray(k_pos)[None, :])
    slot = np.arange(N)
    seen = (slot >= np.asarray(begin)[:, None]) & (slot < np.asarray(end)[:, None])
    p, lse = np.zeros((n, N)), np.full(n, -np.inf)
    for i in range(n):
        if seen[i].any():
            top = t[i, seen[i]].max()
            w = np.exp(t[i, seen[i]] - top)
            p[i, seen[i]] = w / w.sum()
            lse[i] = top + np.log(w.sum())
    return p @ np.where(seen.any(0)[:, None], v, 0.0), p, lse


def evict(weights, n, keep, sink, recent):
    """The slots that stay of one sequence-head's n tokens, ascending."""
    if n <= keep:
        return np.arange(n)
    middle = np.arange(sink, n - recent)
    w = np.where(np.isnan(weights[middle]), -np.inf, weights[middle].astype(np.float64))
    nan = np.isnan(weights[middle])
    best = middle[np.lexsort((middle, nan, -w))][:keep - sink - recent]
    return np.concatenate([np.arange(sink), np.sort(best), np.arange(n - recent, n)])
