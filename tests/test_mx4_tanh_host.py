"""The fraction that stands for tanh in the MXFP4 products' SiTU-GLU: its coefficients, read from the kernel's source,
evaluated as the kernel does, against tanh (no GPU needed)."""
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_latent_moe_amd", "csrc")


@pytest.fixture(scope="module")
def fraction():
    """Coefficients of numerator and denominator, highest power of x^2 first."""
    with open(os.path.join(CSRC, "mx4.hip")) as f:
        body = re.search(r"void tanh_ratio\(.*?\n}", f.read(), re.S)[0]
    start = re.search(r"float p = (\S+)f, q = (\S+)f;", body)
    c = [[float(start[i])] + [float(v) for v in re.findall(rf"fmaf\({n}, t, (\S+?)f\)", body)] for i, n in ((1, "p"), (2, "q"))]
    assert [len(v) for v in c] == [5, 5] and "-9.0f), 9.0f)" in body
    return [np.array(v).astype(np.float32) for v in c]


X = np.concatenate([np.linspace(1e-6, 9, 400001), np.geomspace(1e-30, 9, 50001)])


def test_exact_arithmetic(fraction):
    p, q = (np.polyval(c.astype(np.float64), X * X) for c in fraction)
    assert np.abs(X * p / q / np.tanh(X) - 1).max() < 4.4e-8
    assert 1 - np.tanh(9.0) < 3.1e-8  # past 9 the argument is held there
    assert 2.0 ** -9 <= q.min() and q.max() <= 1  # the range that SiTU-GLU's shared division counts on


def test_fp32(fraction):
    """Every step rounded to fp32, the division aside: an fma's product of two fp32 numbers is exact in float64."""
    x = np.unique(X.astype(np.float32))
    t = x * x

    def horner(c):
        v = np.full_like(t, c[0])
        for k in c[1:]:
            v = (v.astype(np.float64) * t + k).astype(np.float32)
        return v

    num, den = x * horner(fraction[0]), horner(fraction[1])
    assert np.abs(num.astype(np.float64) / den / np.tanh(x.astype(np.float64)) - 1).max() < 3.1e-7
