"""Rotary angles (fmha_rope) of large frequencies at the farthest positions, against exact fractions."""
import math
from fractions import Fraction

import pytest
import torch

from tests import cache_util as cu
from tests.test_rope_gpu import fm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
PI = Fraction(314159265358979323846264338327950288419716939937510582, 10 ** 53)     # off by 10^-53


def test_large_frequencies(fm):  # noqa: F811
    """A turn is off by 2^-24 at most for frequencies up to 2^11: with elements of 1 and 0 the outputs are the cosine and the sine."""
    freq = [2047.9, 1500.123, 700.7, 100.01, 2 * math.pi, 3.1, 1.0, 0.123456789]
    pos = [2 ** 31 - 1, 2 ** 31 - 12345, 1999999999, 1234567890, 2 ** 20 + 1, 77]
    x = torch.zeros((len(pos), 1, 16), dtype=torch.float16)
    x[..., :8] = 1.0
    y, _ = fm.rope(x.cuda(), None, torch.tensor(freq, dtype=torch.float64, device="cuda"),
                   positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    turn = [[float(2 * PI * ((p * Fraction(f) / (2 * PI)) % 1)) for f in freq] for p in pos]
    want = torch.tensor([[math.cos(t) for t in row] + [math.sin(t) for t in row] for row in turn], dtype=torch.float64)
    # the angle: 2^-24 of a turn; sine and cosine 2^-22 more; and f16's half step
    tol = 2 * math.pi * 2.0 ** -24 + 2.0 ** -22
    cu.close(cu.f64(y.cpu())[:, 0], want, tol + (want.abs() + tol) * cu.HALF["f16"], "cosines and sines")
