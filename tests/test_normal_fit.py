"""The polynomials behind the GELU kernels: their errors as the source states
them, and no further from the best possible than rounding to FP32 leaves them. CPU only."""
import math
import os
import re

import numpy as np
import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fft_block_toeplitz_amd", "csrc",
                      "sequence.hpp")


def coefficients(name):
    text = re.search(r"constexpr float %s\[\] = \{(.*?)\};" % name, open(HEADER).read(), re.S).group(1)
    return np.array([np.float32(v.strip().rstrip("f")) for v in text.split(",")], dtype=np.float64)


def tail(k):
    """exp(x^2) erfc(x) / t at t = 1 / (1 + k x)."""
    one = np.vectorize(lambda x: math.exp(x * x) * math.erfc(x))
    return lambda t: one((1.0 / t - 1.0) / k) / t


def centre(u):
    """(Phi(z) - 1/2) / z at u = z^2."""
    z = np.sqrt(np.maximum(u, 1e-12))
    return 0.5 * np.vectorize(math.erf)(z / math.sqrt(2.0)) / z


CASES = [  # name, function, range of its argument, the stated error
    ("kTail16", tail(0.33), (1.0 / (1.0 + 0.33 * 10.0), 1.0), 1.2e-7),
    ("kTail32", tail(0.4), (1.0 / (1.0 + 0.4 * 11.4), 1.0 / (1.0 + 0.4 * math.sqrt(0.5))), 1.3e-7),
    ("kCentre32", centre, (0.0, 1.0), 5.3e-8),
]


@pytest.mark.parametrize("name,function,ends,stated", CASES)
def test_polynomials_are_as_good_as_stated(name, function, ends, stated):
    t = np.linspace(*ends, 20001)
    assert np.abs(np.polyval(coefficients(name)[::-1], t) / function(t) - 1.0).max() < stated * 1.01


@pytest.mark.parametrize("name,function,ends,stated", CASES)
def test_the_fit_is_the_best_of_its_degree(name, function, ends, stated):
    """Least relative error by Lawson's iteration: least squares on Chebyshev
    nodes whose weights are multiplied by the errors until these are level."""
    lo, hi = ends
    n = len(coefficients(name))
    s = -np.cos(np.linspace(0.0, np.pi, 2000))
    rows = np.polynomial.chebyshev.chebvander(s, n - 1) / function(lo + (hi - lo) * (s + 1.0) / 2.0)[:, None]
    weight = np.ones_like(s)
    for _ in range(300):
        root = np.sqrt(weight)
        best = np.abs(rows @ np.linalg.lstsq(rows * root[:, None], root, rcond=None)[0] - 1.0)
        weight *= best / (weight * best).mean()
    # coefficients rounded to FP32 add up to 2^-25 of what they multiply
    assert best.max() <= stated and stated <= best.max() + 2.0 ** -24
