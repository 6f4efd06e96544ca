"""The rotation's sines and cosines at near and far positions against 60-digit decimals."""

from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from quantised_kv_cache_gb300 import tq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantised_kv_cache_gb300 import build
    build.build()


@pytest.mark.parametrize("base", [10000.0, 500000.0, 37.3])
@pytest.mark.parametrize("start", [0, 1 << 20, -1 << 31, (1 << 31) - 300])
def test_sines_and_cosines_at_every_position(base, start):
    """The vector (1, 0) of every pair turns into its cosine and sine. Their error is the last rounding (2^-25 below 1), the one before (a number
    below 1/2: 2^-26), those of the square and the coefficients (2^-24 of at most 0.31 each, 2^-25 together) and the angle's (2^-32 + 2^-34
    turns, 2^-29): below 2^-23, wherever the position is."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    ctx = tq.Context(128, 8, "Q8", 1)
    tq.tq_set_rope(ctx.handle, 128, base=base)
    n = 300
    pos = start + np.arange(n)
    x = torch.zeros(1, 1, n, 128, device=DEV)
    x[..., :64] = 1.0
    y = tq.tq_rotary(ctx.handle, x, torch.as_tensor(pos[None], dtype=torch.int32, device=DEV)).double().cpu().numpy()[0, 0]
    for i in (0, 1, 2, 5, 20, 63):
        f = (-(Decimal(2 * i) / 128) * Decimal(base).ln()).exp() / two_pi
        a = np.array([float((Decimal(int(p)) * f) % 1) for p in pos]) * 2 * np.pi
        assert np.abs(y[:, i] - np.cos(a)).max() <= 2.0 ** -23
        assert np.abs(y[:, 64 + i] - np.sin(a)).max() <= 2.0 ** -23
    ctx.close()
