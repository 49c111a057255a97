"""Bounds of the epilogue's activations on a float32 value that is exact (a
fold of zero weights and a bias): only the evaluation's own rounding, so that a
wrong tail shows."""
from __future__ import annotations

import numpy as np

import operator_refs as refs
from q4_q8_integer_amd import binding

U = refs.U32
# float32's normal range ends here: a result below it may be flushed, and so may
# sigmoid (x < -87.3), which loses up to |v| of it; from |v| = 104 on the result
# itself is below the least float32
FLOOR = 2.0 ** -126


def bound(v: np.ndarray, act: int) -> np.ndarray:
    """The most act(v), v float32 exact, may be off, in float64.  In half steps
    (U) relative to the result:
    SiLU: exp one ulp (2, and a share e / (1 + e) <= 1 of it), 1 + e 1, the
    reciprocal one ulp (2), the product 1: 6.
    GELU (tanh): the same of x = 2u, whose roundings (the square's factor 2,
    product 1, fma 1, factor 2: 6) move sigmoid by |x| (1 - sigmoid(x)) of
    themselves.
    GELU: erfc two ulps (4), the products 2; z = -v / sqrt(2) with its constant
    2, which erfc's logarithmic derivative times z amplifies, |2 z
    exp(-z^2) / (sqrt(pi) erfc(z))| <= 2 z^2 + 2 for z > 0 and <= 1 below."""
    v = v.astype(np.float64)
    a = np.abs(refs.act64(v, act))
    flush = FLOOR * (1 + np.minimum(np.abs(v), 104.0))
    if act == binding.ACT_SILU:
        return 6 * U * a + flush
    if act == binding.ACT_GELU_TANH:
        x = 2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
        return (6 + 6 * np.abs(x) * refs._sigmoid(-x)) * U * a + flush
    if act == binding.ACT_GELU:
        return (6 + 2 * np.where(v < 0, v * v + 2, 1.0)) * U * a + FLOOR
    return np.zeros_like(a)


def values(act: int) -> np.ndarray:
    """float32 over both tails and near 0, as far down as the result is a normal
    float32 and a little beyond."""
    low = {binding.ACT_SILU: -110.0, binding.ACT_GELU: -13.4, binding.ACT_GELU_TANH: -11.0}.get(act, -50.0)
    near = np.linspace(-2, 2, 401)
    tiny = np.array([0.0, -0.0, 1e-30, -1e-30, 2.0 ** -149, -(2.0 ** -149), 2.0 ** -126, -(2.0 ** -126)])
    far = np.array([3e38, -3e38, 1e20, -1e20, 200.0, -200.0])
    return np.concatenate([np.linspace(low, 0, 2000), near, np.linspace(0, 40, 400), tiny, far]).astype(np.float32)


def off(got: np.ndarray, v: np.ndarray, act: int) -> np.ndarray:
    """Where got is outside the bound."""
    with np.errstate(over="ignore", invalid="ignore"):
        ref = refs.act64(v.astype(np.float64), act)
        return ~(np.abs(got.astype(np.float64) - ref) <= bound(v, act) * (1 + 1e-5))
