"""The range check of the orthogonalisation's coefficients on the host: a step's largest singular value and
largest |b l + c l^2| against a dense search in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import blockwise_fp8_gemm_amd as pf

OK, VALUE = 0, 8


def accepted(triples):
    """Whether the call takes these steps (an empty matrix: nothing is launched)."""
    d = (pf.NewtonSchulzDesc * 1)(pf.NewtonSchulzDesc(None, 0, 64, 64, None, 64))
    c = (ctypes.c_float * (3 * len(triples)))(*[v for t in triples for v in t])
    st = pf.lib().puro_fp8_newton_schulz_grouped(0, d, 1, len(triples), c, 1e-7, None, 0, None)
    assert st in (OK, VALUE)
    return st == OK


def reach(triples, points=200001):
    """(largest singular value, largest |b l + c l^2|) over the steps, from singular values in [0, 1] on."""
    top, most, widest = 1.0, 0.0, 0.0
    for a, b, c in np.float32(triples).astype(np.float64):
        s = np.linspace(0, top, points)
        top = float(np.abs(s * (a + s * s * (b + c * s * s))).max())
        most, widest = max(most, top), max(widest, float(np.abs(s * s * (b + c * s * s)).max()))
    return most, widest


@pytest.mark.parametrize("c", [1e-30, -1e-30, 1e-12, -1e-12, 1e-8, 1e-38, 0.0])
def test_small_quintic_coefficient(c):
    """(a, -a, c): f turns at l = 1 / 3 and reaches 0.385 a, however small c is."""
    assert not accepted([(6.0, -6.0, c)]) and not accepted([(30.0, -30.0, c)])
    assert accepted([(5.0, -5.0, c)])
    # the second step's range follows from the first one's largest value, 1.92
    assert accepted([(5.0, -5.0, c), (1.0, 0.0, 0.0)]) and not accepted([(5.0, -5.0, c), (1.1, 0.0, 0.0)])


def test_against_a_search():
    rng = np.random.default_rng(3)
    yes = no = 0
    for _ in range(3000):
        steps = rng.integers(1, 4)
        t = [(rng.uniform(-6, 6), rng.uniform(-9, 9), rng.uniform(-9, 9) * 10.0 ** rng.uniform(-12, 0))
             for _ in range(steps)]
        most, widest = reach(t, 2001)
        if abs(most - 2) < 1e-3 or abs(widest - 32) < 1e-2:
            continue       # nearer to a limit than the search resolves
        want = most <= 2 and widest <= 32
        assert accepted(t) == want, (t, most, widest)
        yes, no = yes + want, no + (not want)
    assert yes > 200 and no > 200


def test_coefficients_of_no_step_or_of_two_kinds():
    g = torch.zeros((16, 16))
    for steps, coef in ((5, ()), (2, ((1, 0, 0), 1.0)), (2, (1.0, (1, 0, 0))), (1, (1, 0)), (3, (1, 0, 0, 0))):
        with pytest.raises(ValueError, match="coefficients"):
            pf.puro_fp8_newton_schulz_grouped([g], steps=steps, coefficients=coef)
