"""The fused norm (q8_quantize_norm, q8_quantize_norm_tiled, residual_norm) on
the GPU: r, h, codes and scale words equal to the 64-bit definition with its
roundings, on every row length class, operand, stride and output."""
import numpy as np
import pytest
import torch

import operator_refs as refs
import oracle
from gpu_helpers import host_ds, note, to_dev
from q4_q8_integer_amd import binding

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _inputs(seed, n, k, y="f32", post=False, gate=None, x_scale=2.0):
    rng = np.random.default_rng([970, seed, n, k])
    a = {"x": (rng.standard_normal((n, k)) * x_scale).astype(np.float32),
         "weight": (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)}
    if y:
        a["y"] = rng.standard_normal((n, k)).astype(np.float16 if y == "f16" else np.float32)
        if post:
            a["y_weight"] = (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)
        if gate == "channel":
            a["gate"] = rng.standard_normal(k).astype(np.float32)
        elif gate == "token":
            a["gate"] = rng.standard_normal((n, k)).astype(np.float32)
    return a


def _same(got, ref, what):
    """Equal but for values whose 64-bit result lies within a sum's rounding
    (k * 2^-53 relative, k <= 2^16: 2^-37) of a float32 border: fewer than one
    in 2^12 can (2^-37 against the step 2^-24), and they are one step off."""
    got, ref = np.asarray(got), np.asarray(ref)
    off = got != ref
    assert off.sum() <= 1 + off.size // 4096, "%s: %d of %d differ" % (what, off.sum(), off.size)
    if off.any():
        step = np.spacing(np.abs(ref[off]).astype(np.float32))
        assert (np.abs(got[off].astype(np.float64) - ref[off]) <= 1.5 * step).all(), what


def _run(a, scale=1.0, tiled=False, what=""):
    n, k = a["x"].shape
    note("norm %s n=%d k=%d tiled=%s %s" % (what, n, k, tiled, sorted(a)))
    dev = {key: to_dev(v) for key, v in a.items()}
    x, weight = dev.pop("x"), dev.pop("weight")
    h = torch.empty(n, k, device=x.device)
    f = binding.quantize_norm_tiled if tiled else binding.quantize_norm
    q, ds, r = f(x, weight, EPS, residual_scale=scale, h=h, **dev)
    h2, r2 = binding.norm(x, weight, EPS, residual_scale=scale, **dev)
    torch.cuda.synchronize()
    rr, rh = refs.norm(a["x"], a["weight"], EPS, a.get("y"), a.get("y_weight"), a.get("gate"), scale)
    _same(r.cpu().numpy(), rr, what + " r")
    # what follows is the definition applied to what was stored
    _, rh = refs.norm(r.cpu().numpy(), a["weight"], EPS)
    _same(h.cpu().numpy(), rh, what + " h")
    assert torch.equal(h, h2) and torch.equal(r, r2)
    rq, rds = oracle.quantize(h.cpu().numpy())
    if tiled:
        assert np.array_equal(q.cpu().numpy().view(np.uint16), oracle.q8_tiles(rq)), what
    else:
        assert np.array_equal(q.cpu().numpy(), rq), what
    assert np.array_equal(host_ds(ds), rds), what
    if "y" not in a:
        assert r is x


@pytest.mark.parametrize("n,k", [(1, 32), (3, 96), (2, 512), (5, 544), (1, 4096), (7, 8192), (3, 11008), (2, 16416),
                                 (2, 28672), (1, 32768), (2, 32800), (1, 65536)])
@pytest.mark.parametrize("y,post,gate", [(None, False, None), ("f32", False, None), ("f16", True, "channel"),
                                         ("f32", True, "token")])
def test_norm_shapes(n, k, y, post, gate):
    _run(_inputs(1, n, k, y, post, gate), 1.0 if y is None else 0.75, what="shape")


@pytest.mark.parametrize("n,k", [(1, 256), (127, 512), (128, 256), (129, 1280), (200, 4096)])
@pytest.mark.parametrize("y", [None, "f16"])
def test_norm_tiles(n, k, y):
    _run(_inputs(2, n, k, y, y is not None, "channel" if y else None), tiled=True, what="tiles")


def test_norm_many_rows():
    _run(_inputs(3, 1500, 1024, "f16", False, "token"), what="many")


def test_norm_zero_rows_and_extremes():
    """A zero row (r = 0: h = 0, codes and words 0), a row that y cancels, tiny
    and huge rows (squares that float32 would lose), one outlier."""
    a = _inputs(4, 6, 256, "f32")
    a["x"][0] = a["y"][0] = 0
    a["y"][1] = -a["x"][1]
    a["x"][2] *= np.float32(1e-25)
    a["y"][2] *= np.float32(1e-25)
    a["x"][3] *= np.float32(1e25)
    a["x"][4, 17] = 1e6
    _run(a, what="extremes")
    q, ds, r = binding.quantize_norm(to_dev(a["x"]), to_dev(a["weight"]), EPS, to_dev(a["y"]))
    torch.cuda.synchronize()
    assert not q[:2].any() and not ds[:2].any() and not r[:2].any()


def test_norm_rounds_codes_at_borders():
    """Rows of a scale's odd half steps, so that h / da lies within float32
    rounding of a .5 border throughout: every code is the oracle's."""
    k = 512
    x = np.tile((2 * np.arange(32) + 1).astype(np.float32) / 2, (4, k // 32))
    x[:, ::32] = 127.0
    a = {"x": x, "weight": np.ones(k, np.float32)}
    _run(a, what="borders")


@pytest.mark.parametrize("y16", [False, True])
def test_norm_strides_in_place_and_guards(y16):
    """x and r as one strided array (in place), y and gate as slices, outputs
    inside guarded buffers."""
    n, k = 9, 320
    a = _inputs(5, n, k, "f16" if y16 else "f32", True, "token")
    rr, rh = refs.norm(a["x"], a["weight"], EPS, a["y"], a["y_weight"], a["gate"], 0.5)
    xb = torch.full((n, k + 64), 7.0, device="cuda:0")
    xs = xb[:, 32:32 + k]
    xs.copy_(to_dev(a["x"]))
    yb = torch.zeros((n, 2 * k), dtype=torch.float16 if y16 else torch.float32, device="cuda:0")
    yb[:, k:] = to_dev(a["y"])
    gb = torch.zeros((n, k + 8), device="cuda:0")
    gb[:, :k] = to_dev(a["gate"])
    note("norm strided in place")
    h, r = binding.norm(xs, to_dev(a["weight"]), EPS, yb[:, k:], to_dev(a["y_weight"]), gb[:, :k], 0.5, r=xs)
    torch.cuda.synchronize()
    assert r is xs and (xb[:, :32] == 7).all() and (xb[:, 32 + k:] == 7).all()
    _same(xs.cpu().numpy(), rr, "in place r")
    _, rh = refs.norm(xs.cpu().numpy(), a["weight"], EPS)
    _same(h.cpu().numpy(), rh, "in place h")


def test_norm_empty():
    w = torch.ones(64, device="cuda:0")
    q, ds, r = binding.quantize_norm(torch.zeros((0, 64), device="cuda:0"), w)
    assert q.shape == (0, 64) and ds.shape == (0, 2) and r.shape == (0, 64)


def test_norm_on_a_side_stream_and_in_a_graph():
    n, k = 33, 1024
    a = _inputs(6, n, k, "f16", True, "channel")
    d = {key: to_dev(v) for key, v in a.items()}
    args = (d["x"], d["weight"], EPS, d["y"], d["y_weight"], d["gate"], 0.5)
    q0, ds0, r0 = binding.quantize_norm(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q1, ds1, r1 = binding.quantize_norm(*args)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(q0, q1) and torch.equal(ds0, ds1) and torch.equal(r0, r1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q2, ds2, r2 = binding.quantize_norm(*args)
    for seed in (7, 8, 9):
        b = _inputs(seed, n, k, "f16", True, "channel")
        d["x"].copy_(to_dev(b["x"]))
        d["y"].copy_(to_dev(b["y"]))
        g.replay()
        q3, ds3, r3 = binding.quantize_norm(*args)
        torch.cuda.synchronize()
        assert torch.equal(q2, q3) and torch.equal(ds2, ds3) and torch.equal(r2, r3)
