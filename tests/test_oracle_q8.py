"""The fp64 restatement of the 8-bit cache (oracle/q8.py) against independent statements: torch's
e4m3 conversion, the scale's defining inequality, small hand-made cases."""

import numpy as np
import pytest
import torch

from oracle import q8


def test_the_grid_is_the_e4m3_numbers():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(q8.GRID, codes)


def test_rounding_equals_torchs_conversion():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g).float())
    mid = torch.from_numpy((q8.GRID[1:] + q8.GRID[:-1]) / 2).float()  # every tie
    x = torch.cat([x.clamp(-448, 448), mid, -mid, torch.tensor([0.0, 448.0, -448.0, 1e-9])])
    want = x.to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(q8.e4m3(x.double().numpy()), want)
    assert q8.e4m3(np.array([np.inf]))[0] == 448.0 and q8.e4m3(np.array([-np.inf]))[0] == -448.0


@pytest.mark.parametrize("amax", [1e-45, 1e-30, 2.0 ** -91.2, 1.0, 1.75, 1.7500001, 447.9, 448.0, 448.1, 3.4e38])
def test_the_exponent_is_the_least(amax):
    e = q8.exponent(amax)
    assert e >= q8.MIN_EXP and amax <= 448 * 2.0 ** e
    assert e == q8.MIN_EXP or amax > 448 * 2.0 ** (e - 1)


def test_a_larger_token_rescales_the_block_and_a_smaller_one_does_not():
    m = q8.Model(1, 128)
    m.append(0, 0, np.full((1, 128), 1.0))
    assert m.exp[0, 0] == -8 and np.all(m.codes[0, 0] == 256)
    m.append(0, 1, np.full((1, 128), 0.5))
    assert m.exp[0, 0] == -8 and np.all(m.values()[0, 1] == 0.5)
    m.append(0, 2, np.full((1, 128), 100.0))
    assert m.exp[0, 0] == -2 and np.all(m.values()[0, :3, 0] == [1.0, 0.5, 96.0])  # 400 lies between 384 and 416: even code
    m.append(0, 64, np.zeros((1, 128)))
    assert m.exp[0, 1] == q8.MIN_EXP


def test_rotation_keeps_length_and_depends_on_the_distance_only():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 128))
    for il in (False, True):
        dots = [(q8.rope(q, [p + 5], 96, il) @ q8.rope(k, [p], 96, il).T).item() for p in (0, 3, 1000)]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-12)
        back = q8.rope(q8.rope(q, [77], 96, il), [77], 96, il, transpose=True)
        np.testing.assert_allclose(back, q, atol=1e-14)


def test_scaled_frequencies_interpolate_slow_pairs_only():
    f = q8.rope_frequencies(128)
    g = q8.rope_frequencies(128, factor=8.0, original_len=8192, low=1.0, high=4.0)
    assert np.all(g[:20] == f[:20]) and np.allclose(g[-8:], f[-8:] / 8) and np.all((g <= f) & (g >= f / 8))
    np.testing.assert_allclose(q8.rope_frequencies(64, factor=4.0), q8.rope_frequencies(64) / 4)


def test_attention_of_small_cases():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 5, 128))
    out, p, lse = q8.attend(q, k, v, np.zeros(5, int), np.arange(1, 6))
    np.testing.assert_allclose(out[0], v[0])
    want = np.exp(q[4] @ k.T / np.sqrt(128))
    np.testing.assert_allclose(out[4], want @ v / want.sum())
    np.testing.assert_allclose(lse[4], np.log(want.sum()))
    out, p, lse = q8.attend(q, k, v, [2] * 5, [2] * 5)
    assert not out.any() and not p.any() and np.all(np.isneginf(lse))


def test_eviction_of_small_cases():
    w = np.array([9, 1, 5, 5, 5, 0, np.nan, 3], dtype=np.float32)
    assert list(q8.evict(w, 8, 8, 0, 0)) == list(range(8))
    assert list(q8.evict(w, 8, 4, 1, 1)) == [0, 2, 3, 7]
    assert list(q8.evict(w, 8, 7, 0, 0)) == [0, 1, 2, 3, 4, 5, 7]
    assert list(q8.evict(w, 5, 2, 0, 2)) == [3, 4]
