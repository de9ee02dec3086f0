"""Frequencies of rotary positions at the ends of their arguments' ranges."""
import ctypes
import math

import pytest

import kimi_delta_attention_12_gb300 as kda


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_12_gb300 import build
    build.build()


@pytest.mark.parametrize("factor", [1e-12, math.exp(-10.0), 1e-3, 0.5, 1.0 - 2.0 ** -40])
def test_a_factor_below_one_leaves_the_magnitude_at_one(factor):
    """0.1 ln(factor) + 1 would be 0 at e^-10 and negative below.  The base keeps what is divided by
    the factor small."""
    _, m = kda.rotary_frequencies(64, 1e38, "by_parts", factor, 4096.0, fast=2.0 ** -60,
                                  slow=2.0 ** -61, device="cpu")
    assert m == 1.0


@pytest.mark.parametrize("factor", [1.0, 1.0 + 2.0 ** -20, 2.0, 8.0, 1e6])
def test_a_factor_above_one_raises_it(factor):
    _, m = kda.rotary_frequencies(64, 1e4, "by_parts", factor, device="cpu")
    assert abs(m - (0.1 * math.log(factor) + 1.0)) <= 2.0 ** -23
