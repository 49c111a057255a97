"""Plain 64-bit references of the epilogue, the router, the combination and the
fused norm, in numpy, and the weight bytes their tests use."""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

import oracle
from q4_q8_integer_amd import binding, synth

U32 = 2.0 ** -24          # half a step of float32, relative
U16 = 2.0 ** -11          # half a step of binary16, relative
SUB16 = 2.0 ** -25        # half a step of binary16 subnormals


def weights(fmt: str, seed: int, m: int, k: int) -> np.ndarray:
    """Random weight rows of format 'q4k' or 'q6k' as uint8 [m, bytes]."""
    if fmt == "q4k":
        return synth.pack_q4k(synth.random_fields(seed, m, k))
    return synth.pack_q6k(synth.random_q6k_fields(seed, m, k))


def fold64(fmt: str, w: np.ndarray, m: int, k: int, q: np.ndarray, ds: np.ndarray) -> np.ndarray:
    return (oracle.out_f64 if fmt == "q4k" else oracle.q6k_out_f64)(w, m, k, q, ds)


def act64(v: np.ndarray, act: int) -> np.ndarray:
    if act == binding.ACT_RELU:
        return np.maximum(v, 0.0)
    if act == binding.ACT_SILU:
        return v * _sigmoid(v)
    if act == binding.ACT_GELU:
        return 0.5 * v * erfc(-v / np.sqrt(2.0))
    if act == binding.ACT_GELU_TANH:
        return v * _sigmoid(2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3))
    return v


def _sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def act_error(v: np.ndarray, act: int) -> np.ndarray:
    """A bound of float32 act(v)'s error, v = fold + bias rounded once
    (relative U32).  Through the activation that rounding becomes at most
    |act'| <= 1.13 times U32 |v|.  The evaluation adds, in units of U32 |act|:
    SiLU: exp 2 (one ulp), 1 + e 1, the division 1 (and 2 to spare);
    GELU: erfc 4, two products 2, and the rounding of z = -v / sqrt(2)
    (constant and product, 2), which erfc's logarithmic derivative, at most
    2 z^2 + 2, amplifies; GELU-tanh: as SiLU, and u's roundings (square 1,
    product 2, fma 1, factor 2: 6) times |2u|, as sigmoid's logarithmic
    derivative times its argument is at most |2u|."""
    a = np.abs(act64(v, act))
    e = 1.13 * np.abs(v)
    if act == binding.ACT_SILU:
        e = e + 6 * a
    elif act == binding.ACT_GELU:
        e = e + (6 + 2 * (v * v + 2)) * a
    elif act == binding.ACT_GELU_TANH:
        e = e + (6 + 6 * np.abs(1.6 * (v + 0.044715 * v ** 3))) * a
    return e * U32


def check_epilogue(got: np.ndarray, fold32: np.ndarray, bias, act: int, residual, f16: bool, what: str = ""):
    """got against the epilogue of the float32 fold in 64 bits, within the
    rounding of the float32 steps (act_error, the residual's addition) and of
    a binary16 store."""
    v = fold32.astype(np.float64) + (0.0 if bias is None else bias.astype(np.float64))
    ref, tol = act64(v, act), act_error(v, act)
    if residual is not None:
        ref = ref + residual.astype(np.float64)
        tol = tol + U32 * (np.abs(ref) + tol)
    if f16:
        tol = tol + U16 * (np.abs(ref) + tol) + SUB16
    # results below float32's normal range may be flushed steps of 2^-149
    err = np.abs(got.astype(np.float64) - ref)
    bad = err > tol * (1 + 1e-6) + 2.0 ** -126
    assert not bad.any(), "%s: %d values off, worst %.3g of its bound" % (
        what, int(bad.sum()), float((err / (tol + 2.0 ** -126)).max()))


def route(logits: np.ndarray, top: int, normalize: bool, scale: float):
    """(ids, weights float64, slot, rows, offsets) of the router, by loops."""
    n, experts = logits.shape
    l = logits.astype(np.float64)
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, float(np.finfo(np.float32).max))
    ids = np.full((n, top), -1, np.int32)
    weights = np.zeros((n, top))
    groups = [[] for _ in range(experts)]
    for t in range(n):
        order = sorted(range(experts), key=lambda e: (-l[t, e], e))
        chosen = [e for e in order if l[t, e] > -np.inf][:top]
        if not chosen:
            continue
        over = chosen if normalize else [e for e in range(experts) if l[t, e] > -np.inf]
        total = sum(np.exp(l[t, e] - l[t, chosen[0]]) for e in over)
        for j, e in enumerate(chosen):
            ids[t, j] = e
            weights[t, j] = scale * np.exp(l[t, e] - l[t, chosen[0]]) / total
            groups[e].append((t, j))
    slot = np.full((n, top), -1, np.int32)
    rows = np.full(n * top, -1, np.int32)
    offsets = [0]
    s = 0
    for group in groups:
        for t, j in group:
            slot[t, j], rows[s] = s, t
            s += 1
        offsets.append(s)
    return ids, weights, slot, rows, np.array(offsets, np.int32)


def norm(x, weight, eps, y=None, y_weight=None, gate=None, scale=1.0):
    """(r float32, h float32) of the fused norm: float64 between the roundings."""
    r = x
    if y is not None:
        z = y.astype(np.float64)
        if y_weight is not None:
            z = z * y_weight.astype(np.float64) / np.sqrt((z * z).mean(1, keepdims=True) + float(np.float32(eps)))
        if gate is not None:
            z = z * gate.astype(np.float64)
        r = (float(np.float32(scale)) * x.astype(np.float64) + z).astype(np.float32)
    rd = r.astype(np.float64)
    h = rd * weight.astype(np.float64) / np.sqrt((rd * rd).mean(1, keepdims=True) + float(np.float32(eps)))
    return r, h.astype(np.float32)
