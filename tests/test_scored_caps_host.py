"""The capping polynomials against tanh on the host: the errors that the sources state for them, and the bound on a score
that decides how far they are used."""
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_scaled_dot_softmax_gb300", "csrc")


@pytest.fixture(scope="module")
def source():
    return open(os.path.join(CSRC, "api_scored.cu")).read()


def numbers(source, name):
    m = re.search(name + r"(?:\[\d\])?\s*=\s*\{?([^;}]*)[};,]", source)
    return [float(x) for x in re.findall(r"-?\d[\d.e+-]*", m.group(1))]


def odd(coefficients, x):
    return x * sum(c * x ** (2 * i) for i, c in enumerate(coefficients))


def test_errors_of_the_fits(source):
    near, wide = numbers(source, "kNear"), numbers(source, "kWide")
    assert len(near) == 3 and len(wide) == 7
    x = np.linspace(1e-6, 0.5, 1_000_001)
    off, t = np.abs(odd(near, x) - np.tanh(x)), np.tanh(x)
    assert (off / x).max() <= 2.2e-5 == numbers(source, "kNearError")[0] and (off / t).max() <= 2.4e-5 and off.max() <= 1.1e-5
    assert np.abs(odd(near, x) ** 2 - t * t).max() <= 1.05e-5
    x = np.linspace(1e-6, 1.7, 1_000_001)
    off, t = np.abs(odd(wide, x) - np.tanh(x)), np.tanh(x)
    assert off.max() <= 8.8e-6 < 9.1e-6 == float(re.search(r"kWideError = ([\d.e-]+)", source).group(1))
    assert (off / x).max() <= 3.6e-5
    assert np.abs(odd(wide, x) ** 2 - t * t).max() <= 1.7e-5
    # the series of the third range, in fp32's place: its first neglected term
    x = np.linspace(1e-6, 0.25, 1_000_001)
    assert np.abs(odd([1, -1 / 3, 2 / 15, -17 / 315, 62 / 2835], x) / np.tanh(x) - 1).max() <= 1e-8


@pytest.mark.parametrize("cap", [1.0, 20.0, 50.0, 54.5, 65.9, 66.0, 100.0, 1000.0, 1e6])
def test_the_fits_are_used_only_within_the_bound(source, cap):
    """With the rule as the source has it: a score is off by at most 6e-4 wherever a fit is taken."""
    bound = numbers(source, "kCapError")[0]
    assert bound == 6e-4
    assert "std::min(0.5, kCapError / (kNearError * form->cap))" in source
    assert "kWideError * form->cap <= kCapError ? 1.7 : 0.0" in source
    near, wide = numbers(source, "kNear"), numbers(source, "kWide")
    x = np.linspace(0, min(0.5, bound / (2.2e-5 * cap)), 100_001)
    assert (cap * np.abs(odd(near, x) - np.tanh(x))).max() <= bound
    if 9.1e-6 * cap <= bound:
        x = np.linspace(0, 1.7, 100_001)
        assert (cap * np.abs(odd(wide, x) - np.tanh(x))).max() <= bound


def test_caps_that_are_refused():
    import ctypes
    import __graft_entry__
    __graft_entry__.build()
    from transformer_scaled_dot_softmax_gb300 import _native as m
    fake = 1 << 20
    for cap, want in ((9e-19, m.MHA_ERR_INVALID_ARG), (1.1e18, m.MHA_ERR_INVALID_ARG), (1e30, m.MHA_ERR_INVALID_ARG),
                      (1e-18, m.MHA_ERR_MISALIGNED), (1e18, m.MHA_ERR_MISALIGNED), (0.0, m.MHA_ERR_MISALIGNED)):
        f = m.ScoreForm()
        f.cap = cap
        # the pointers' alignment is checked after the form
        assert m.lib.sdpa_scored_forward(1, fake + 2, fake, fake, fake, None, None, None, 0, 1, 2, 2, 8, 8, 64, 64, 0.125, 0, None,
                                         ctypes.addressof(f), None, None) == want, cap
