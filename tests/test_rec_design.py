"""What the recurrence's kernels rely on, checked on the CPU."""
import os
import random
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_depthwise_conv1d_gb300", "csrc")


def test_tile_places_by_multiplication_are_exact():
    """t / n as the high half of 2 t (2^63 / n + 1), for tiles below 2^31."""
    rng = random.Random(1)
    cases = [(t, n) for n in (1, 2, 3, 7, 64, 80, 641, 2 ** 20 + 7, 2 ** 31 - 1) for t in (0, 1, n - 1, n, 2 * n - 1, 2 ** 31 - 1)]
    cases += [(rng.randrange(2 ** 31), rng.randrange(1, 2 ** rng.randrange(1, 32))) for _ in range(20000)]
    for t, n in cases:
        if t < 2 ** 31 and 1 <= n < 2 ** 31:
            inv = 2 ** 63 // n + 1
            assert inv < 2 ** 64
            assert (2 * t * inv) >> 64 == t // n, (t, n)


def coefficients():
    text = open(os.path.join(CSRC, "glr.cuh")).read()
    block = re.search(r"float c\[7\] = \{(.*?)\};", text, re.S).group(1)
    return [float.fromhex(v.strip().rstrip("f")) if "x" in v else float(v.strip().rstrip("f")) for v in block.split(",")]


def test_the_polynomial_of_expm1_over_its_range():
    c = coefficients()
    x = np.linspace(-0.85, -1e-6, 200001)
    p = np.zeros_like(x)
    for v in c:
        p = p * x + v
    # the fit 8e-10; six coefficients rounded to FP32 (half of 2^-24 each) enter with 0.85, 0.85^2 / 2 .. of 0.67 to 1
    assert np.abs(p * x / np.expm1(x) - 1).max() < 2.0 ** -25
    # in FP32, each step rounded once.  u = 2^-24: the steps' values, at most 1, 0.5, 0.17, 0.04 .. from the last back, enter
    # the result times 1, 0.85, 0.85^2 ..: 1.6 u of a result of at least 0.67, 2.4 u; the coefficients' own roundings
    # (none in the last) 0.5 u; the product with l u.  Together less than 4 u
    x32 = x.astype(np.float32)
    p = np.full_like(x32, c[0])
    for v in c[1:]:
        p = (p.astype(np.float64) * x32 + v).astype(np.float32)
    e = (p * x32).astype(np.float64)
    assert np.abs(e / np.expm1(x32.astype(np.float64)) - 1).max() < 4 * 2.0 ** -24


def test_statistics_from_a_shift_lose_little():
    """A thread's squares about its mean from sums about the mean of its first vector, in FP32: values with an outlying
    first vector, and with a large common mean."""
    rng = np.random.default_rng(2)
    for n, lead, base in ((10, 0.0, 0.0), (16, 1e4, 0.0), (64, 3e5, 0.0), (16, 0.0, 3e3)):
        x = (rng.standard_normal((n, 8)) + base).astype(np.float32)
        x[0] += np.float32(lead)
        shift = np.float32(x[0].sum(dtype=np.float32) / 8)
        d = (x - shift).astype(np.float32)
        s = q = np.float32(0)
        for v in d.ravel():
            s = np.float32(s + v)
            q = np.float32(np.float64(v) * v + q)
        off = np.float32(s / (8 * n))
        m2 = np.float32(np.float64(q) - np.float64(off) * off * 8 * n)
        exact = ((x.astype(np.float64) - x.astype(np.float64).mean()) ** 2).sum()
        # n / 8 V of the sum's own error: 8 n roundings of the sum of squares about the shift
        assert abs(m2 / exact - 1) < (8 * n + 8) * n * 2.0 ** -24


@pytest.mark.parametrize("name", ["glr_fwd.cu", "glr_bwd.cu", "gn_cluster.cu"])
def test_waits_that_run_out_are_recorded(name):
    """No wait's result is dropped, except of those that only wait for copies in flight before a block ends."""
    text = open(os.path.join(CSRC, name)).read()
    for m in re.finditer(r"!mbar_wait\(|!glr_look_back\(", text):
        assert "g_fault" in text[m.start():m.start() + 250], text[m.start():m.start() + 80]
    for m in re.finditer(r"(?<!!)\bmbar_wait\(", text):
        assert "in flight" in text[m.start():m.start() + 120]
