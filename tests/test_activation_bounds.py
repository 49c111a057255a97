"""The bounds that the activations are held to catch what a looser one let
pass: a tail of zeros, 1 + erf in place of erfc, and an exponential of a
rounded x * log2(e)."""
import numpy as np
import pytest
from scipy.special import erf, erfc

import activation_bounds as ab
import operator_refs as refs
from q4_q8_integer_amd import binding

F = np.float32
ACTS = [binding.ACT_SILU, binding.ACT_GELU, binding.ACT_GELU_TANH]


def model(v, act, exp):
    """The float32 steps of out.h with numpy's correctly rounded operations."""
    with np.errstate(over="ignore", under="ignore"):
        if act == binding.ACT_GELU:
            z = (F(-0.70710678118654752) * v).astype(F)
            return ((F(0.5) * v) * erfc(z.astype(np.float64)).astype(F)).astype(F)
        x = v
        if act == binding.ACT_GELU_TANH:
            s = ((F(0.044715) * v) * v).astype(F).astype(np.float64) * v + v
            x = (F(1.59576912160573076) * s.astype(F)).astype(F)
        return v * (F(1) / (F(1) + exp(-x)))


def exact_exp(x):
    return np.exp(x.astype(np.float64)).astype(F)


def exp2_of_rounded(x):
    return np.exp2((F(1.44269504088896341) * x).astype(np.float64)).astype(F)


@pytest.mark.parametrize("act", ACTS)
def test_the_definition_in_float32_is_within(act):
    v = ab.values(act)
    got = model(v, act, exact_exp)
    assert not ab.off(got, v, act).any()


@pytest.mark.parametrize("act", ACTS)
def test_a_tail_of_zeros_is_not(act):
    v = ab.values(act)
    got = model(v, act, exact_exp)
    for cut in (-1.0, -4.0, -8.0):
        zero = np.where(v < cut, F(0), got)
        tail = (v < cut) & (v > -9.8)   # where the exact value is a normal float32 in every form
        assert ab.off(zero, v, act)[tail].all(), cut


def test_one_plus_erf_is_not():
    v = ab.values(binding.ACT_GELU)
    with np.errstate(under="ignore"):
        got = (F(0.5) * v) * (F(1) + erf((F(0.70710678118654752) * v).astype(np.float64)).astype(F))
    assert ab.off(got, v, binding.ACT_GELU)[(v < -4) & (v > -13)].mean() > 0.9


def test_an_exponential_of_a_rounded_product_is_not():
    v = ab.values(binding.ACT_SILU)
    got = model(v, binding.ACT_SILU, exp2_of_rounded)
    assert ab.off(got, v, binding.ACT_SILU)[(v < -20) & (v > -80)].mean() > 0.25
