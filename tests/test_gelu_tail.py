"""The polynomial behind gelu in the products' epilogue, from its coefficients in the
source, against exp(x^2) erfc(x) in 64 bits, and what gelu's error is made of."""
import os
import re

import numpy as np
import pytest

special = pytest.importorskip("scipy.special")
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_03_gb300", "csrc",
                      "fused.cuh")
U = 2.0 ** -24


def body():
    with open(SOURCE) as f:
        text = f.read()
    start = text.index("F2 normal_cdf(F2 z, F2& e) {")
    return text[:start], text[start:text.index("\n}\n", start)]


def tail(x):
    """t P(t) of the source, and x"""
    code = body()[1]
    p = [float(c) for c in re.findall(r"0\.5f \* (-?[0-9.]+)f", code)]
    slope = float(re.search(r"fma2\(F2\(([0-9.]+)f\), a,", code).group(1))
    assert len(p) == 8
    t = 1 / (1 + slope * np.sqrt(2) * x)
    return t * np.polyval(p, t)


def test_the_polynomial_is_as_good_as_its_comment_says():
    x = np.linspace(0, 10, 1000001)
    worst = np.abs(tail(x) / special.erfcx(x) - 1).max()
    said = float(re.search(r"relative error \(([0-9.e-]+) up to x = 10\)", body()[0]).group(1))
    assert 0.9 * said < worst <= said


def test_gelu_in_32_bits():
    # The kernel's operations one by one in FP32.  Relative to z times the distribution: the polynomial 3.9e-7 (6.6 U); its
    # evaluation 8 U at most, as its terms are of one size; exp's argument is off by 1.5 U of z^2 / 2 and its constant by as
    # much, together 1.5 z^2 U; ex2, rcp (2^-22, or 4 U, each in the kernel, less here) and the products 12 U.
    F = np.float32
    z = np.linspace(-12, 12, 200001).astype(F)
    code = body()[1]
    p = [F(0.5) * F(c) for c in re.findall(r"0\.5f \* (-?[0-9.]+)f", code)]
    slope = F(re.search(r"fma2\(F2\(([0-9.]+)f\), a,", code).group(1))
    e = np.exp2((z * z * F(-0.72134752044448170368)).astype(np.float64)).astype(F)
    t = (1 / (slope * np.abs(z) + F(1)).astype(np.float64)).astype(F)
    q = np.full_like(t, p[0])
    for c in p[1:]:
        q = q * t + c
    q = q * t * e
    got = z * np.where(z < 0, q, F(1) - q)
    want = z.astype(np.float64) * special.ndtr(z.astype(np.float64))
    bound = (1.5 * z.astype(np.float64) ** 2 + 6.6 + 8 + 12) * U * np.abs(want) + 1e-30
    assert (np.abs(got - want) <= bound).all()
