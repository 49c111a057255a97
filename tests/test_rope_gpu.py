"""Rotary positions on the GPU against the formula in extended precision."""
import numpy as np
import pytest
import torch

import attention_refs as refs
from gpu_helpers import note, to_dev
from q4_q8_integer_amd import binding as b

pytestmark = pytest.mark.gpu


def _freq(pairs, theta=1e4):
    return (theta ** (-np.arange(pairs) / pairs)).astype(np.float32)


def _check(got, x, ref, half, what):
    # float64 to some 1e-15 of the pair's magnitude, a rounding to float32, one to the type
    a = 2.0 ** -48 * np.abs(x.astype(np.float64)).max() * 4
    refs.check(got, ref, refs.U32 * np.abs(ref) + a, half, what)


@pytest.mark.parametrize("n,heads,dim,pairs", [(1, 1, 2, 1), (1, 32, 128, 64), (3, 2, 5, 2), (7, 3, 80, 40), (5, 4, 96, 24),
                                               (2, 1, 1024, 512), (33, 5, 6, 3), (4, 8, 64, 20), (9, 2, 40, 8),
                                               (300, 4, 128, 32), (6, 1, 257, 100)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
def test_rope(n, heads, dim, pairs, half, adjacent):
    rng = np.random.default_rng([11, n, dim])
    x = rng.standard_normal((n, heads * dim)).astype(np.float16 if half else np.float32)
    pos = rng.integers(0, 100000, (n, 1)).astype(np.int32)
    f = _freq(pairs)
    ref = refs.rope(x, heads, pos, f, adjacent=adjacent)
    note("rope n=%d heads=%d dim=%d pairs=%d" % (n, heads, dim, pairs))
    d = to_dev(x)
    got = b.rope(d, heads, b.Rope(to_dev(pos[:, 0]), to_dev(f), None, adjacent))
    torch.cuda.synchronize()
    assert np.array_equal(d.cpu().numpy(), x)
    _check(got.cpu().numpy(), x, ref, half, "rope")
    assert b.rope(d, heads, b.Rope(to_dev(pos), to_dev(f), None, adjacent), out=d) is d
    assert torch.equal(d, got)


@pytest.mark.parametrize("axes", [1, 2, 3, 5])
def test_axes_scale_and_far_positions(axes):
    rng = np.random.default_rng([12, axes])
    n, heads, dim, pairs = 12, 3, 64, 32
    x = rng.standard_normal((n, heads * dim)).astype(np.float32)
    pos = rng.integers(-2 ** 31, 2 ** 31, (n, axes)).astype(np.int32)
    pos[0], pos[1], pos[2] = 0, 2 ** 31 - 1, -2 ** 31
    f = _freq(pairs)
    f[3], f[4] = 0.0, -1.5
    axis = rng.integers(-2, axes + 2, pairs).astype(np.int32)      # out of range counts as the nearest
    ref = refs.rope(x, heads, pos, f, axis, scale=1.25)
    wide = torch.zeros(n, axes + 3, dtype=torch.int32, device="cuda:0")
    wide[:, :axes] = to_dev(pos)
    got = b.rope(to_dev(x), heads, b.Rope(wide[:, :axes], to_dev(f), to_dev(axis), False, 1.25))
    torch.cuda.synchronize()
    _check(got.cpu().numpy(), x, ref, False, "axes")


@pytest.mark.parametrize("half", [False, True])
def test_strides(half):
    rng = np.random.default_rng(13)
    n, heads, dim, pairs = 5, 2, 32, 16
    for extra in (8, 3):                                            # the second leaves the 16-byte grid
        wide = to_dev(rng.standard_normal((n, heads * dim + extra)).astype(np.float16 if half else np.float32))
        x = wide[:, :heads * dim]
        pos, f = to_dev(np.arange(n, dtype=np.int32) * 7), to_dev(_freq(pairs))
        want = b.rope(x.contiguous(), heads, b.Rope(pos, f))
        before = wide.clone()
        b.rope(x, heads, b.Rope(pos, f), out=x)
        torch.cuda.synchronize()
        assert torch.equal(x, want) and torch.equal(wide[:, heads * dim:], before[:, heads * dim:])


@pytest.mark.parametrize("adjacent", [False, True])
def test_rows_on_16_byte_boundaries_alone(adjacent):
    """Float32 rows that begin 16 bytes past a 32-byte boundary, and at a stride
    of an odd number of 16 bytes."""
    rng = np.random.default_rng(14)
    n, heads, dim, pairs = 6, 2, 48, 16
    flat = to_dev(rng.standard_normal(4 + n * (heads * dim + 4)).astype(np.float32))
    x = flat[4:].view(n, heads * dim + 4)[:, :heads * dim]
    assert x.data_ptr() % 32 == 16 and x.stride(0) % 8 == 4
    pos, f = to_dev(rng.integers(0, 5000, n).astype(np.int32)), to_dev(_freq(pairs))
    was = x.cpu().numpy().copy()
    b.rope(x, heads, b.Rope(pos, f, None, adjacent), out=x)
    torch.cuda.synchronize()
    _check(x.cpu().numpy(), was, refs.rope(was, heads, pos.cpu().numpy(), f.cpu().numpy(), adjacent=adjacent), False, "rope")


def test_non_finite_values_stay_in_their_pair():
    x = torch.ones(2, 64, device="cuda:0")
    x[0, 5], x[1, 40] = float("nan"), float("inf")
    got = b.rope(x, 1, b.Rope(to_dev(np.array([3, 4], np.int32)), to_dev(_freq(32))))
    bad = ~torch.isfinite(got).cpu()
    assert bad[0].nonzero().flatten().tolist() == [5, 37] and bad[1].nonzero().flatten().tolist() == [8, 40]


def test_empty_and_refusals():
    dev = "cuda:0"
    f, pos = torch.ones(4, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    assert b.rope(torch.zeros(0, 16, device=dev), 2, b.Rope(pos[:0], f)).shape == (0, 16)
    x = torch.zeros(3, 16, device=dev)
    for bad in (lambda: b.rope(x, 3, b.Rope(pos, f)), lambda: b.rope(x, 2, b.Rope(pos[:2], f)),
                lambda: b.rope(x, 2, b.Rope(pos, f, torch.zeros(5, dtype=torch.int32, device=dev))),
                lambda: b.rope(x, 2, b.Rope(pos.long(), f)), lambda: b.rope(x.double(), 2, b.Rope(pos, f)),
                lambda: b.rope(x, 2, b.Rope(pos, f.half())), lambda: b.rope(x, 2, b.Rope(pos.cpu(), f)),
                lambda: b.rope(x, 2, None), lambda: b.rope(x, 2, b.Rope(pos, f), out=x.half()),
                lambda: b.rope(x, 2, b.Rope(pos, torch.ones(5, device=dev)))):
        with pytest.raises((TypeError, ValueError, b.MMQError)):
            bad()
