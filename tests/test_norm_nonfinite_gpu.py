"""NaN and infinities through the fused norm: they stay visible in the codes'
scale words and in every product of their token, and change no other token."""
import numpy as np
import pytest
import torch

import operator_refs as refs
import oracle
from gpu_helpers import host_ds, note, to_dev
from q4_q8_integer_amd import binding

pytestmark = pytest.mark.gpu
NAN, INF = np.nan, np.inf


def _words_nan(ds):
    return np.isnan((ds & 0xFFFF).astype(np.uint16).view(np.float16))


def _inputs(k, seed=1):
    rng = np.random.default_rng([971, seed, k])
    x, y = (rng.standard_normal((10, k)).astype(np.float32) for _ in range(2))
    x[1, k // 3] = NAN
    x[2, k - 1] = INF
    y[3, 0] = NAN
    y[4, k // 2] = -INF
    x[6, 5], y[6, 5] = INF, -INF                 # a NaN of their own
    x[7] = NAN
    x[8], y[8] = 3e38, 3e38                      # the new stream overflows float32, unless y is normed to about 1
    return x, y, (1 + 0.2 * rng.standard_normal(k)).astype(np.float32), rng.standard_normal(k).astype(np.float32)


def _split(post):
    """The finite rows and the others."""
    good = [0, 5, 9] + ([8] if post else [])
    return good, [i for i in range(10) if i not in good]


@pytest.mark.parametrize("k", [256, 4096, 16640, 33024])          # a value per lane, two, four, and passes
@pytest.mark.parametrize("post,gate", [(False, False), (True, True)])
@pytest.mark.parametrize("tiled", [False, True])
def test_norm_keeps_nonfinite_tokens_visible(k, post, gate, tiled):
    x, y, w, g = _inputs(k)
    note("norm nonfinite k=%d post=%s tiled=%s" % (k, post, tiled))
    kw = dict(y_weight=to_dev(w) if post else None, gate=to_dev(g) if gate else None)
    f = binding.quantize_norm_tiled if tiled else binding.quantize_norm
    h = torch.empty(10, k, device="cuda:0")
    q, ds, r = f(to_dev(x), to_dev(w), 1e-5, to_dev(y), h=h, **kw)
    h2, r2 = binding.norm(to_dev(x), to_dev(w), 1e-5, to_dev(y), **kw)
    torch.cuda.synchronize()
    good, bad = _split(post)
    h, r, ds = h.cpu().numpy(), r.cpu().numpy(), host_ds(ds)
    assert np.array_equal(h, h2.cpu().numpy(), equal_nan=True) and np.array_equal(r, r2.cpu().numpy(), equal_nan=True)
    assert np.isfinite(h[good]).all() and np.isfinite(r[good]).all()
    assert not np.isfinite(r[bad]).all(1).any()
    # a block's scale is NaN where its h has one, and each bad token has such a block
    blocks = np.isnan(h).reshape(10, k // 32, 32).any(2)
    assert np.array_equal(_words_nan(ds), blocks) and blocks[bad].any(1).all()
    # the other tokens are the quantizer's
    rq, rds = oracle.quantize(np.where(np.isfinite(h), h, 0))
    assert np.array_equal(ds[good], rds[good])
    if not tiled:
        assert np.array_equal(q.cpu().numpy()[good], rq[good])


@pytest.mark.parametrize("tiled", [False, True])
def test_norm_nan_in_a_weight_and_a_zero_row_without_eps(tiled):
    k = 512
    x, _, w, _ = _inputs(k, 2)
    x = np.where(np.isfinite(x), x, 1).astype(np.float32)
    w[70] = NAN
    f = binding.quantize_norm_tiled if tiled else binding.quantize_norm
    note("norm nan weight")
    _, ds, _ = f(to_dev(x), to_dev(w))
    torch.cuda.synchronize()
    nan = _words_nan(host_ds(ds))
    assert nan[:, 2].all() and not np.delete(nan, 2, axis=1).any()
    x[3] = 0
    w[70] = 1
    _, ds, _ = f(to_dev(x), to_dev(w), 0.0)      # 0 / 0
    torch.cuda.synchronize()
    nan = _words_nan(host_ds(ds))
    assert nan[3].all() and not np.delete(nan, 3, axis=0).any()


def _fold(fmt, w, m, k, q, ds, bias):
    return binding.fold_epilogue(fmt, w, m, k, q, ds, bias, binding.ACT_SILU)


# every kernel behind the fold: dot4, stream, narrow, few, binary16, and the repacked, tiled and q6_K ones
@pytest.mark.parametrize("fmt,m,n", [(binding.FORMAT_Q4K, 14340, 1), (binding.FORMAT_Q4K, 14340, 4),
                                     (binding.FORMAT_Q4K, 14340, 12), (binding.FORMAT_Q4K, 200, 7),
                                     (binding.FORMAT_Q4K, 200, 16), (binding.FORMAT_Q4K, 5000, 12),
                                     (binding.FORMAT_Q4K, 200, 40), (binding.FORMAT_Q4K, 200, 150),
                                     (binding.FORMAT_Q4K_REPACKED, 200, 13), (binding.FORMAT_Q4K_REPACKED, 200, 100),
                                     (binding.FORMAT_Q4K_TILES, 200, 60), (binding.FORMAT_Q4K_REPACKED_TILES, 200, 140),
                                     (binding.FORMAT_Q6K, 200, 6), (binding.FORMAT_Q6K, 200, 30),
                                     (binding.FORMAT_Q6K, 5000, 30), (binding.FORMAT_Q6K, 5000, 10),
                                     (binding.FORMAT_Q6K, 33000, 70), (binding.FORMAT_Q6K_TILES, 200, 60)])
def test_products_of_nonfinite_tokens_are_nan(fmt, m, n):
    k = 4096
    rng = np.random.default_rng([972, fmt, m, n])
    x = rng.standard_normal((n, k)).astype(np.float32)
    bad = np.zeros(n, bool)
    bad[::3] = True
    x[bad, rng.integers(0, k, bad.sum())] = np.where(np.arange(bad.sum()) % 2, NAN, -INF)
    fix = np.where(bad[:, None], np.float32(0), x)
    w = to_dev(refs.weights("q6k" if fmt in (binding.FORMAT_Q6K, binding.FORMAT_Q6K_TILES) else "q4k", n, m, k).reshape(-1))
    if fmt in (binding.FORMAT_Q4K_REPACKED, binding.FORMAT_Q4K_REPACKED_TILES):
        w = binding.repack(w, m, k)
    f = binding.quantize_norm_tiled if fmt in binding._TILE_FORMATS else binding.quantize_norm
    one, bias = torch.ones(k, device="cuda:0"), torch.randn(m, device="cuda:0")
    note("fold nonfinite fmt=%d m=%d n=%d" % (fmt, m, n))
    got, ref = (_fold(fmt, w, m, k, *f(to_dev(a), one)[:2], bias) for a in (x, fix))
    torch.cuda.synchronize()
    got, ref = got.cpu().numpy(), ref.cpu().numpy()
    assert np.isnan(got[bad]).all() and np.isfinite(ref).all()
    assert np.array_equal(got[~bad], ref[~bad])


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
def test_grouped_products_of_nonfinite_tokens_are_nan(fmt):
    """Through both few-token forms and the binary16 kernels, and combined: a
    bad token is NaN, the tokens that share its experts are not."""
    m, k, n, top, experts = 136, 512, 60, 3, 6
    rng = np.random.default_rng([973, len(fmt)])
    x = rng.standard_normal((n, k)).astype(np.float32)
    bad = np.zeros(n, bool)
    bad[[0, 7, 8, 30, 59]] = True
    fix = x.copy()
    x[bad, 11] = [NAN, INF, -INF, NAN, INF]
    one = torch.ones(k, device="cuda:0")
    w = to_dev(np.concatenate([refs.weights(fmt, 40 + e, m, k).reshape(-1) for e in range(experts)]))
    f = binding.FORMAT_Q4K if fmt == "q4k" else binding.FORMAT_Q6K
    logits = rng.standard_normal((n, experts)).astype(np.float32) + np.array([4, 0, 1, -1, -2, 0], np.float32)
    rt = binding.route(to_dev(logits), top)
    note("grouped nonfinite %s" % fmt)
    outs = []
    for a in (x, fix):
        q, ds, _ = binding.quantize_norm(to_dev(a), one)
        y = binding.fold_grouped(f, w, experts, m, k, q, ds, rt.offsets, rt.rows)
        outs.append((y.cpu().numpy(), binding.combine(y, rt.slot, rt.weights).cpu().numpy()))
    sizes = np.diff(rt.offsets.cpu().numpy())
    assert sizes.min() <= 16 < sizes.max()
    at = bad[rt.rows.cpu().numpy()]
    (y, out), (yr, outr) = outs
    assert np.isnan(y[at]).all() and np.array_equal(y[~at], yr[~at]) and np.isfinite(yr).all()
    assert np.isnan(out[bad]).all() and np.array_equal(out[~bad], outr[~bad])
