"""Attention over the cache where few tokens have nearly all of the weight and
the others nearly all of the output (what a product of weight and scale loses
goes by the largest such product, not by the largest weight), and queries
whose smallest values count."""
import numpy as np
import pytest
import torch

import attention_refs as refs
from gpu_helpers import note
from q4_q8_integer_amd import binding as b
from test_kv_attend_gpu import Case

pytestmark = pytest.mark.gpu


def put(c, t, k, k_scale, v, v_scale):
    """Token t of the one sequence and head: codes and a scale for all blocks."""
    dim, bits = c.dim, c.bits
    parts, cb, sb = refs.record_parts(dim, c.page, bits), dim * bits // 8, dim // 16
    rec = c.data[c.table[0, t // c.page], 0]
    for code, scale, at, place, whole in ((k, k_scale, 0, refs.key_place(dim), c.k), (v, v_scale, 2, refs.value_place(dim), c.v)):
        d = np.float16(scale)
        assert np.abs(code).max() <= (127 if bits == 8 else 7)
        rec[parts[at] + t % c.page * cb:][:cb] = refs.code_bytes(code, place, bits, at == 0)
        rec[parts[at + 1] + t % c.page * sb:][:sb] = np.full(dim // 32, d).view(np.uint8)
        whole[0][0, t] = code * np.float64(d)


def sink(dim, bits, group, length, gap, half, v_scale=2.0 ** -24, tokens=(0,), width=None):
    """Rows of ones over `length` tokens of scores near 0 and positive values,
    but for `tokens` with scores `gap` above them and values of v_scale."""
    c = Case(80, 1, group, dim, 64, bits, [length], [1], half, width=width)
    rng = np.random.default_rng([80, dim, bits, length])
    lim = 127 if bits == 8 else 7
    c.q[:] = 1
    for t in range(length):
        if t in tokens:
            put(c, t, np.full(dim, lim), gap / (lim * dim), np.full(dim, lim), v_scale)
        else:
            put(c, t, rng.integers(-lim, lim + 1, dim), 1 / (lim * dim), rng.integers(lim // 2 + 1, lim + 1, dim), 1 / lim)
    return c


def check(c, full, window=0):
    """Within the bounds of every rounding; the floor of the products is, for
    each token, 2^-29 of the largest product of a weight and its token's largest
    value.  (A reference lies 2^5 below a product of weight and 2^e, which bounds a
    scale within a factor of 2; half a step of binary16 is 2^-25 there and a code
    127 at most: 2^-29 of a product whose code is 127.  A scale of 0 counts as 2^-64.)"""
    out, lse = c.run(window, 1.0)
    torch.cuda.synchronize()
    k, v, length = c.k[0][0], c.v[0][0], int(c.lengths[0])
    lo = max(0, length - window) if window else 0
    s = k.sum(-1)[lo:]
    w = np.exp(s - s.max())
    total = w.sum()
    w, v = w / total, v[lo:]
    ref = w @ v
    lim = 127 if c.bits == 8 else 7
    size = np.maximum(np.abs(v).max(-1), lim * 2.0 ** -64)
    floor = len(s) * 2.0 ** -29 * (w * size).max()
    tol = refs.bound_of(np.abs(k[lo:]).sum(-1), s, w, v, ref, full) - len(s) * 2.0 ** -27 * np.abs(v).max() + floor
    got = out.cpu().numpy()[0].reshape(c.group, c.dim)
    for row in got:
        refs.check(row, ref, tol, out.dtype == torch.float16)
    want = s.max() + np.log(total)
    assert (np.abs(lse.cpu().numpy() - want) <= 2e-4 + 4e-7 * abs(want)).all()
    return tol / np.abs(ref)


@pytest.mark.parametrize("group", [2, 40, 200])               # every form's rows
@pytest.mark.parametrize("dim,bits", [(32, 8), (128, 8), (128, 4), (160, 8)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("length,gap", [(300, 16.0), (1200, 19.0)])
def test_a_token_with_the_weight_and_no_value(group, dim, bits, half, length, gap):
    note("sink dim=%d bits=%d group=%d length=%d gap=%g half=%d" % (dim, bits, group, length, gap, half))
    worst = check(sink(dim, bits, group, length, gap, half), not half)
    assert worst.max() < 4e-3                                  # the bound says something


@pytest.mark.parametrize("tokens", [(5,), (299,), (2, 40, 170, 290), (31, 32, 33)])
@pytest.mark.parametrize("group", [1, 40])
def test_such_tokens_anywhere(tokens, group):
    check(sink(64, 8, group, 300, 19.0, False, tokens=tokens), True)


@pytest.mark.parametrize("gap", [40.0, 55.0])
@pytest.mark.parametrize("group", [1, 200])
def test_far_above_the_others(gap, group):
    """The tokens without a value have all of the weight that float32 knows of."""
    check(sink(32, 8, group, 400, gap, False, v_scale=0.0), True)


def test_long_flat_tail():
    """99.9% of the weight on a first token of small values, over 40000 others."""
    worst = check(sink(32, 8, 2, 40000, float(np.log(999 * 40000)), False, v_scale=2.0 ** -20), True)
    assert worst.max() < 4e-3


@pytest.mark.parametrize("group", [1, 200])
@pytest.mark.parametrize("fall", [True, False])
def test_scores_that_fall_and_rise(group, fall):
    """Scores from 60 to -60 along the cache, or back; the values grow against them."""
    c = Case(81, 1, group, 32, 64, 8, [640], [1])
    c.q[:] = 1
    rng = np.random.default_rng(81)
    for t in range(640):
        u = t if fall else 639 - t
        s = 60 - 120 * u / 639
        put(c, t, np.full(32, 100 if s > 0 else -100), abs(s) / 3200, rng.integers(64, 128, 32),
            0.0 if u < 32 else 2.0 ** (-14 + 28 * u / 639))
    k, v = c.k[0], c.v[0]
    out, lse = c.run(0, 1.0)
    torch.cuda.synchronize()
    ref, l, tol = refs.attend(c.q.reshape(1, group, 32), k, v, np.ones(640, bool), 639, group, 1.0, 0)
    refs.check(out.cpu().numpy(), ref.reshape(1, -1), tol.reshape(1, -1), False)
    rel = np.abs(out.cpu().numpy() - ref.reshape(1, -1)) / np.abs(ref.reshape(1, -1))
    # sums of magnitudes: 152 steps of scores up to 60, and of weights 32 a step of 640 tokens
    assert rel.max() <= 2.0 ** -24 * (2 * 152 * 64 + 4 * 64) + 2.0 ** -20
    assert (np.abs(lse.cpu().numpy()[0] - l) <= 2e-4 + 4e-7 * np.abs(l)).all()


def test_rows_keep_their_bits_beside_others():
    """A row's references move by its own scores: beside rows whose scores rise
    elsewhere it gives the same bits."""
    c = Case(82, 1, 3, 64, 64, 8, [700], [1])
    c.q[0, 64:128] *= 8
    alone, l1 = c.run()
    c.q[0, :64] = 0
    c.q[0, 128:] *= 20
    beside, l2 = c.run()
    torch.cuda.synchronize()
    assert torch.equal(alone[0, 64:128], beside[0, 64:128]) and l1[0, 1] == l2[0, 1]


@pytest.mark.parametrize("group", [1, 24, 130])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("spread", [8.0, 40.0])
def test_peaked_scores_beside_scales_of_any_size(group, half, spread):
    """Random keys, values and scales, with scores up to some hundred: a row's
    largest products move from token to token."""
    Case(83, 1, group, 64, 64, 8, [900, 260], [1, 1], half, spread=spread).both(most=1)


@pytest.mark.parametrize("group", [1, 40, 200])
@pytest.mark.parametrize("out_half", [False, True])
@pytest.mark.parametrize("large", [8192.0, 16384.0, 32768.0, 65504.0])
@pytest.mark.parametrize("small", [1, 3, 1023])
def test_binary16_queries_are_exact(group, out_half, large, small):
    """Scores that the smallest values of a head make beside its largest one."""
    c = Case(84, 1, group, 32, 16, 8, [3], [1], True)
    c.q[0].reshape(group, 32)[:, :] = 0
    c.q[0].reshape(group, 32)[:, 0] = large
    c.q[0].reshape(group, 32)[:, 1] = small * 2.0 ** -24
    for t, code in enumerate((127, 0, -127)):
        k = np.zeros(32, np.int64)
        k[1] = code
        put(c, t, k, 1 / 64, np.arange(32) + 45 * t, 1 / 64)
    out, lse = c.run(0, 2.0 ** 24 / small, f16=out_half)
    torch.cuda.synchronize()
    c.check(out, lse, scale=2.0 ** 24 / small, half=out_half)


@pytest.mark.parametrize("base", [1e3, 1e5, 7e5, 1.4e6, 2.8e6, 5.5e6])
@pytest.mark.parametrize("half", [False, True])
def test_far_scores_beside_scales_of_any_size(base, half):
    """Scores whose float32 steps come near those of their differences, over values
    of 2^-14 to 2^9: what comes out lies among the values."""
    c = Case(85, 1, 200, 64, 64, 8, [1200], [1], half)
    rng = np.random.default_rng([85, int(base)])
    parts, q = refs.record_parts(64, 64, 8), np.zeros((200, 64))
    q[:, :32] = base / (32 * 127) * (1 + 0.2 * rng.random((200, 1)))
    q[:, 32] = 0.5 + rng.random(200)
    c.q[:] = q.reshape(1, -1)
    for t in range(1200):
        k = np.full(64, 127, np.int64)
        k[32:] = 0
        k[32] = rng.integers(-127, 128)
        put(c, t, k, 1.0, rng.integers(64, 128, 64), 2.0 ** rng.uniform(-21, 2))
        c.data[c.table[0, t // 64], 0, parts[1] + t % 64 * 4 + 2:][:2] = np.full(1, 0.1, np.float16).view(np.uint8)
    out, lse = c.run(0, 1.0)
    torch.cuda.synchronize()
    got, v = out.cpu().numpy().reshape(200, 64).astype(np.float64), c.v[0][0]
    assert np.isfinite(got).all() and torch.isfinite(lse).all()
    # weights are positive and sum up to 1 but for roundings: 2^-11 each, sums of 1200
    assert (got <= v.max(0) * (1 + 2.0 ** -9)).all() and (got >= v.min(0) * (1 - 2.0 ** -9) - 2.0 ** -24).all()
