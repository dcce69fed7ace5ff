"""Options that fp32, in which the kernels work, cannot hold are refused on the host
(no device work: what is accepted ends at a workspace that is too small)."""
import ctypes

import pytest

from linear_cross_entropy_tile_amd import flce

A = 0x1000
ACCEPTED, BAD_OPTION = 5, 9


def _process(which, **kw):
    o = flce.FlceProcessOptions()
    for k, v in {**dict(ignore_index=-100, repetition_penalty=1.0, temperature=1.0,
                        logits_dtype=1, out_dtype=1), **kw}.items():
        setattr(o, k, v)
    if which == "forward":
        return flce.lib().flce_process_logits(A, 10, 4, 10, ctypes.byref(o), 2 * A, 10, None, None,
                                              None, A, 0, None)
    g = flce.FlceProcessGrads(2 * A, 10, None, None, None, 0, None, None)
    return flce.lib().flce_process_logits_backward(ctypes.byref(g), A, 10, 4, 10, ctypes.byref(o),
                                                   3 * A, 10, A, 0, None)


@pytest.mark.parametrize("which", ["forward", "backward"])
@pytest.mark.parametrize("name", ["repetition_penalty", "temperature"])
@pytest.mark.parametrize("value,code", [
    # 1e-46 would be 0, for a temperature "unscaled"; 1e-40 has no reciprocal in fp32.
    (1e-46, BAD_OPTION), (1e-320, BAD_OPTION), (1e-40, BAD_OPTION), (2.0 ** -128, BAD_OPTION),
    (1e39, BAD_OPTION), (1e300, BAD_OPTION),
    (2.0 ** -127, ACCEPTED), (1e-30, ACCEPTED), (0.7, ACCEPTED), (3e38, ACCEPTED)])
def test_divisors_of_logits(which, name, value, code):
    assert _process(which, **{name: value}) == code


@pytest.mark.parametrize("which", ["forward", "backward"])
def test_a_temperature_of_zero_is_no_divisor(which):
    assert _process(which, temperature=0.0) == ACCEPTED
    assert _process(which, repetition_penalty=0.0) == BAD_OPTION


@pytest.mark.parametrize("softcap,code", [
    # Of 1e-40 the reciprocal is infinite in fp32, and a logit of 0 would be NaN.
    (1e-40, 6), (2.0 ** -128, 6), (1e-44, 6), (2.0 ** -127, ACCEPTED), (1e-20, ACCEPTED),
    (50.0, ACCEPTED), (3e38, ACCEPTED), (0.0, ACCEPTED), (-1e-40, ACCEPTED)])
def test_tanh_cap_of_logits(softcap, code):
    assert flce.lib().flce_logits(A, A, None, 4, 8, 10, softcap, 1, A, 10, A, 0, None) == code


@pytest.mark.parametrize("eps,code", [
    # In fp32 these are 0 or denormals: a gradient of 0 would make its weight 0 / 0.
    (1e-320, BAD_OPTION), (1e-50, BAD_OPTION), (1e-40, BAD_OPTION), (2.0 ** -127, BAD_OPTION),
    (2.0 ** -126, ACCEPTED), (1e-30, ACCEPTED), (1e-8, ACCEPTED), (0.0, ACCEPTED)])
def test_eps_of_adamw(eps, code):
    o = flce.FlceAdamwOptions(1e-3, 0.9, 0.999, eps, 0.01, flce.FLCE_STATE_F32,
                              flce.FLCE_ROUND_NEAREST, 0)
    table = flce.FlceAdamwList()
    assert flce.lib().flce_adamw_step(ctypes.byref(table), ctypes.byref(o), None, None, A, A, 0,
                                      None) == code
