"""The norm's root next to the borders where fp32 rounds the other way."""
import math
import random
from fractions import Fraction

import numpy as np
import pytest

from tests.test_step_gpu import DEV, tq2  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def squares(S, rng):
    """Eight whole numbers below 2^24 whose squares add up to S (about 2^48.6), or None."""
    x, rest = [], S
    for most in (1 << 23, 1 << 23, 1 << 23):
        x.append(rng.randint(1 << 22, most))
        rest -= x[-1] ** 2
    x.append(math.isqrt(rest // 2))
    rest -= x[-1] ** 2
    for _ in range(4):
        x.append(math.isqrt(rest))
        rest -= x[-1] ** 2
    return x if rest == 0 and max(x) < 1 << 24 else None


def rows(n, seed):
    """Rows of eight whole numbers, exact in fp32, whose 1/sqrt(mean of squares)
    lies 2^-50 to 2^-47 beside the middle between two neighbours in fp32, and
    what it rounds to."""
    rng = random.Random(seed)
    x, r = [], []
    while len(x) < n:
        low = np.float32(rng.uniform(2.0 ** -22.9, 2.0 ** -22.7))
        high = np.nextafter(low, np.float32(1))
        middle = (Fraction(float(low)) + Fraction(float(high))) / 2
        up = rng.random() < 0.7
        # a smaller sum has a larger root
        S = round(8 / middle ** 2 * (1 - Fraction(rng.uniform(0.5, 2) * (1 if up else -1)) / 2 ** 47))
        one = next(filter(None, (squares(S, rng) for _ in range(1000))), None)
        if one is None:
            continue
        assert (Fraction(S, 8) < 1 / middle ** 2) == up
        rng.shuffle(one)
        x.append(one)
        r.append(high if up else low)
    return np.array(x, np.float32), np.array(r, np.float32)


def test_root_next_to_borders(tq2):  # noqa: F811
    x, r = rows(200, 1)
    out, _ = tq2.tq2_add_rms_norm(torch.from_numpy(x).to(DEV), eps=0.0, out_dtype=torch.float32)
    got = out.cpu().numpy()
    want = x * r[:, None]
    assert want.dtype == np.float32
    wrong = np.flatnonzero((got != want).any(1))
    assert len(wrong) == 0, len(wrong)
    q, s, _ = tq2.tq2_add_rms_norm_i8(torch.from_numpy(x).to(DEV), eps=0.0)
    assert np.array_equal(s.cpu().numpy(), np.abs(want).max(1) / np.float32(127))
