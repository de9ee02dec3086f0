"""Frequencies of rotary positions at the ends of their arguments' ranges."""
import ctypes
import math

import pytest
import torch

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


@pytest.mark.parametrize("base,scaling,factor,ok", [
    (2.0 ** -20, 0, 1.0, True),              # the largest is 2^(20 * 62 / 64)
    (2.0 ** -21, 0, 1.0, False), (1e-300, 0, 1.0, False), (5e-324, 0, 1.0, False),
    (1e4, 1, 2.0 ** -19, True), (1e4, 1, 2.0 ** -20, False), (1e4, 1, 1e-300, False),
    (1e4, 2, 1e-30, False), (1e308, 2, 1e-300, False),
])
def test_frequencies_that_the_rotary_call_does_not_take_are_refused(base, scaling, factor, ok):
    f, m = (ctypes.c_float * 32)(*[7.0] * 32), ctypes.c_float(7.0)
    st = kda.lib().kda_rotary_frequencies(64, base, scaling, factor, 4096.0, 32.0, 1.0,
                                          ctypes.addressof(f), ctypes.addressof(m))
    if ok:
        assert st == kda.KDA_OK and max(f) < 2.0 ** 20 and m.value == 1.0
    else:
        assert st == kda.KDA_ERR_INVALID_ARG and list(f) == [7.0] * 32 and m.value == 7.0


@pytest.mark.parametrize("device,to", [(None, "cuda"), (0, 0), (1, 1), ("cpu", "cpu"),
                                       (torch.device("cpu"), torch.device("cpu"))])
def test_frequencies_go_to_the_device_that_is_named(monkeypatch, device, to):
    """Device 0 is device 0, whichever is the current one."""
    seen = []
    monkeypatch.setattr(torch.Tensor, "to", lambda self, where: seen.append(where) or self)
    kda.rotary_frequencies(64, device=device)
    assert seen == [to]
