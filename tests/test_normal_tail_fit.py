"""The polynomials of GELU's normal tail (csrc/act.cu): the fit that gave them, and
the error of what stands in the source, in 64 bits and with every operation rounded
to fp32."""
import math
import os
import re

import numpy as np
import pytest

from conftest import ROOT

Y_MAX = 14.5
F = np.float32


def _source(which):
    """(k, coefficients) as act.cu has them for results in fp32 or bf16."""
    text = open(os.path.join(ROOT, "fp4_precision_gemms_gb300", "csrc", "act.cu")).read()
    body = text[text.index("NormalTail normal_tail("):]
    k = re.search(r"constexpr float k = (?:FAST \? ([\d.]+)f : )?([\d.]+)f;", body)
    c = re.search(r"constexpr float %s\[\] = \{(.*?)\};" % ("full" if which == "fp32" else "fast"), body, re.S).group(1)
    return F(k.group(2 if which == "fp32" else 1)), np.array([F(v) for v in re.findall(r"-?[\d.]+(?=f)", c)])


def _scaled(y):
    """exp(y^2 / 2) Phi(-y)."""
    return np.array([0.5 * math.exp(v * v / 2) * math.erfc(v * 0.5 ** 0.5) for v in y])


def fit(k, degree, points=4000, rounds=400):
    """Q of t (1/2 + w Q(w)), t = 1 / (1 + k y), w = 1 - t: least squares of the relative
    error at Chebyshev's points of w, each round weighted by the errors of the one before
    (Lawson's algorithm); the best round's (error, coefficients)."""
    top = k * Y_MAX / (1 + k * Y_MAX)
    w = 0.5 * top * (1 + np.cos((np.arange(points) + 0.5) * np.pi / points))
    g = _scaled(w / (k * (1 - w))) / (1 - w)
    a = np.stack([w ** (i + 1) / g for i in range(degree + 1)], 1)
    b = (g - 0.5) / g
    weight, best = np.ones(points), (np.inf, None)
    for _ in range(rounds):
        c = np.linalg.lstsq(a * weight[:, None] ** 0.5, b * weight ** 0.5, rcond=None)[0]
        error = np.abs(a @ c - b)
        if error.max() < best[0]:
            best = error.max(), c
        weight = weight * np.sqrt(error / error.max()) + 1e-12
        weight /= weight.sum()
    return best


CASES = [("fp32", 8, 2e-8, 4e-8, 4e-7), ("bf16", 6, 3e-7, 3e-7, 5e-6)]  # polynomial's degree, its error, with rounded coefficients, the tail's


@pytest.mark.parametrize("which,degree,fitted,rounded,whole", CASES)
def test_fit(which, degree, fitted, rounded, whole):
    k, c = _source(which)
    assert len(c) == degree + 1
    error, own = fit(float(k), degree)
    assert error <= fitted
    y = np.linspace(0, Y_MAX, 20001)
    t = 1 / (1 + float(k) * y)
    g = _scaled(y) / t
    value = lambda q: 0.5 + (1 - t) * np.polyval(np.asarray(q, float)[::-1], 1 - t)  # noqa: E731
    assert np.abs(value(c) / g - 1).max() <= rounded
    assert np.abs(value(own) / value(c) - 1).max() <= rounded + fitted


def _fma(a, b, c):
    return F(np.float64(a) * np.float64(b) + np.float64(c))


@pytest.mark.parametrize("which,degree,fitted,rounded,whole", CASES)
def test_every_operation_rounded(which, degree, fitted, rounded, whole):
    """The tail as the kernel computes it, with an exponential to nearest."""
    k, c = _source(which)
    y = np.linspace(0, 12.9, 40001).astype(F)
    ky = F(k * y)
    t = F(1) / F(F(1) + ky)
    w = F(ky * t) if which == "fp32" else F(F(1) - t)
    q = np.full_like(y, c[-1])
    for a in c[-2::-1]:
        q = _fma(q, w, a)
    yy = F(y * y)
    e = F(np.exp(np.float64(F(-0.5) * yy)))
    if which == "fp32":
        e = _fma(e, F(-0.5) * _fma(y, y, -np.float64(yy)), e)
    tail = F(e * F(t * _fma(w, q, 0.5)))
    want = np.array([0.5 * math.erfc(v * 0.5 ** 0.5) for v in y.astype(np.float64)])
    assert np.abs(tail / want - 1).max() <= whole
