"""The router and the combination on the GPU against loops in 64 bits, and a
feed-forward block of experts as a user runs it: norm and quantize, route,
grouped gate and up, SiLU quantize, grouped down, combine; eager and captured."""
import numpy as np
import pytest
import torch

import operator_refs as refs
import oracle
from gpu_helpers import host_ds, note, to_dev
from q4_q8_integer_amd import binding, synth

pytestmark = pytest.mark.gpu


def _check_route(logits, top, normalize=True, scale=1.0, dev=None):
    note("route n=%d experts=%d top=%d" % (logits.shape[0], logits.shape[1], top))
    r = binding.route(to_dev(logits) if dev is None else dev, top, normalize, scale)
    torch.cuda.synchronize()
    ids, weights, slot, rows, offsets = refs.route(logits, top, normalize, scale)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.slot.cpu().numpy(), slot)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    # exp: one ulp (2 half steps) and the rounding of l - max, |l - max| <= 2^5
    # where its weight counts: 2^5 half steps; the sum's terms alike, its
    # additions log2(1024) + 6, the division and the scale 2
    got = r.weights.cpu().numpy().astype(np.float64)
    assert (np.abs(got - weights) <= 100 * refs.U32 * weights + 2.0 ** -126).all()
    return r


@pytest.mark.parametrize("n,experts,top", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (5, 64, 8), (7, 65, 1), (4, 100, 64),
                                           (16, 128, 8), (130, 60, 6), (33, 200, 7), (9, 257, 8), (6, 1024, 10),
                                           (700, 16, 4), (2100, 8, 2)])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_shapes(n, experts, top, normalize):
    rng = np.random.default_rng([991, n, experts])
    logits = (rng.standard_normal((n, experts)) * 3).astype(np.float32)
    _check_route(logits, top, normalize, 1.0 if normalize else 2.5)


def test_route_ties_masks_and_extremes():
    rng = np.random.default_rng(992)
    logits = rng.integers(-2, 3, (40, 90)).astype(np.float32)        # many ties
    logits[3] = 1.0                                                   # all equal
    logits[4] = -np.inf                                               # a padding row
    logits[5, 1:] = -np.inf                                           # one expert left
    logits[6, ::2] = -np.inf
    logits[7, :5] = np.nan                                            # NaN masks
    logits[8] = np.nan
    logits[9, 3] = np.inf                                             # +inf: the largest float
    logits[9, 70] = np.inf
    logits[10, 7] = np.finfo(np.float32).max
    logits[11, 9] = np.finfo(np.float32).min                          # the lowest value is not a mask
    logits[12] = np.finfo(np.float32).min
    logits[13] = -np.inf
    logits[13, [80, 2]] = [-1e38, 3e38]
    for top in (1, 4, 64):
        for normalize in (True, False):
            _check_route(logits, top, normalize)
    _check_route(np.full((5, 6), -np.inf, np.float32), 2)            # no slots at all


def test_route_strided_and_empty():
    rng = np.random.default_rng(993)
    wide = rng.standard_normal((20, 50)).astype(np.float32)
    dev = to_dev(wide)[:, :37]
    _check_route(np.ascontiguousarray(wide[:, :37]), 3, dev=dev)
    r = binding.route(torch.zeros((0, 8), device="cuda:0"), 2)
    assert r.ids.shape == (0, 2) and r.rows.shape == (0,) and not r.offsets.any()


def test_route_refusals():
    l = torch.zeros(4, 8, device="cuda:0")
    for top in (0, 9, -1):
        with pytest.raises(ValueError):
            binding.route(l, top)
    with pytest.raises(TypeError):
        binding.route(l.half(), 2)
    with pytest.raises(ValueError):
        binding.route(torch.zeros(8, 4, device="cuda:0").t(), 2)
    with pytest.raises(binding.MMQError):
        binding.route(torch.zeros(2, 1025, device="cuda:0"), 2)


@pytest.mark.parametrize("n,m,top,f16,residual", [(1, 1, 1, False, False), (3, 7, 2, True, True), (5, 64, 8, True, False),
                                                  (17, 4096, 2, False, True), (4, 100, 3, False, True),
                                                  (9, 1032, 4, True, True), (2, 11008, 64, False, False),
                                                  (300, 12, 6, True, False)])
def test_combine(n, m, top, f16, residual):
    rng = np.random.default_rng([994, n, m])
    slots = n * top + 3
    y = rng.standard_normal((slots, m)).astype(np.float16 if f16 else np.float32)
    slot = rng.permutation(slots)[:n * top].reshape(n, top).astype(np.int32)
    slot[rng.random((n, top)) < 0.2] = -1
    slot[-1] = -1                                                     # a token without any expert
    if n > 2:
        slot[1, 0] = slots                                            # past the end counts as none
    y[np.setdiff1d(np.arange(slots), slot)] = np.nan                  # what no token takes is not read into the sum
    wt = rng.random((n, top)).astype(np.float32)
    r = rng.standard_normal((n, m)).astype(np.float32) if residual else None
    note("combine n=%d m=%d top=%d" % (n, m, top))
    out = binding.combine(to_dev(y), to_dev(slot), to_dev(wt), None if r is None else to_dev(r))
    torch.cuda.synchronize()
    live = (slot >= 0) & (slot < slots)
    terms = np.where(live[:, :, None], wt[:, :, None].astype(np.float64) * y[np.where(live, slot, 0)].astype(np.float64), 0)
    ref = terms.sum(1) + (0 if r is None else r)
    # one rounding per fma and one for the residual, each at most half a step of
    # the largest partial sum
    tol = refs.U32 * (top + 1) * (np.abs(terms).sum(1) + (0 if r is None else np.abs(r)))
    assert (np.abs(out.cpu().numpy() - ref) <= tol * (1 + 1e-6)).all()
    if r is not None:
        inplace = to_dev(r)
        got = binding.combine(to_dev(y), to_dev(slot), to_dev(wt), inplace, inplace)
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_combine_refusals():
    y, s, w = torch.zeros(8, 16, device="cuda:0"), torch.zeros(4, 2, dtype=torch.int32, device="cuda:0"), None
    w = torch.zeros(4, 2, device="cuda:0")
    with pytest.raises(ValueError):
        binding.combine(y, s, w[:, :1].contiguous())
    with pytest.raises(TypeError):
        binding.combine(y, s.long(), w)
    with pytest.raises(TypeError):
        binding.combine(y.double(), s, w)
    with pytest.raises(ValueError):
        binding.combine(y, s, w, torch.zeros(4, 15, device="cuda:0"))


class Block:
    """A feed-forward block of experts."""

    def __init__(self, n, k, ff, experts, top, seed):
        rng = np.random.default_rng([995, seed])
        self.n, self.k, self.ff, self.experts, self.top = n, k, ff, experts, top
        self.gate_w = [refs.weights("q4k", 100 + e, ff, k) for e in range(experts)]
        self.up_w = [refs.weights("q4k", 200 + e, ff, k) for e in range(experts)]
        self.down_w = [refs.weights("q6k", 300 + e, k, ff) for e in range(experts)]
        cat = lambda ws: to_dev(np.concatenate([w.reshape(-1) for w in ws]))  # noqa: E731
        self.d = [cat(self.gate_w), cat(self.up_w), cat(self.down_w)]
        self.router = to_dev((rng.standard_normal((experts, k)) / np.sqrt(k)).astype(np.float32))
        self.weight = to_dev((1 + 0.1 * rng.standard_normal(k)).astype(np.float32))

    def run(self, x, y):
        b, (gw, uw, dw) = binding, self.d
        h = torch.empty_like(x)
        q, ds, r = b.quantize_norm(x, self.weight, 1e-5, y, h=h)
        rt = b.route((h[:, None, :] * self.router).sum(-1), self.top)
        gate = b.fold_grouped(b.FORMAT_Q4K, gw, self.experts, self.ff, self.k, q, ds, rt.offsets, rt.rows)
        up = b.fold_grouped(b.FORMAT_Q4K, uw, self.experts, self.ff, self.k, q, ds, rt.offsets, rt.rows)
        hq, hds = b.quantize_silu_mul(gate, up)
        # float32: with weights of this size the outputs reach 1e5, past binary16's 65504
        down = b.fold_grouped(b.FORMAT_Q6K, dw, self.experts, self.k, self.ff, hq, hds, rt.offsets)
        return {"h": h, "q": q, "ds": ds, "r": r, "rt": rt, "gate": gate, "up": up, "hq": hq, "hds": hds, "down": down,
                "out": b.combine(down, rt.slot, rt.weights, r)}

    def check(self, o):
        """Every step against 64 bits on the inputs that the step before gave."""
        host = lambda t: t.cpu().numpy()  # noqa: E731
        q, ds = oracle.quantize(host(o["h"]))
        assert np.array_equal(host(o["q"]), q) and np.array_equal(host_ds(o["ds"]), ds)
        rt = o["rt"]
        off, rows = host(rt.offsets), host(rt.rows)
        assert off[-1] == self.n * self.top
        hq, hds = oracle.quantize_silu_mul(host(o["gate"]), host(o["up"]))
        assert np.array_equal(host(o["hq"]), hq) and np.array_equal(host_ds(o["hds"]), hds)
        for e in range(self.experts):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            for name, w in (("gate", self.gate_w), ("up", self.up_w)):
                ref = refs.fold64("q4k", w[e], self.ff, self.k, q[rows[a:b]], ds[rows[a:b]])
                got = host(o[name])[a:b]
                assert np.linalg.norm(got - ref) <= 1e-5 * np.linalg.norm(ref)
            ref = refs.fold64("q6k", self.down_w[e], self.k, self.ff, hq[a:b], hds[a:b])
            assert np.linalg.norm(host(o["down"])[a:b] - ref) <= 1e-5 * np.linalg.norm(ref)
        slot, wt = host(rt.slot), host(rt.weights).astype(np.float64)
        ref = host(o["r"]) + (wt[:, :, None] * host(o["down"]).astype(np.float64)[slot]).sum(1)
        assert np.linalg.norm(host(o["out"]) - ref) <= 1e-6 * np.linalg.norm(ref)


@pytest.mark.parametrize("n", [1, 6, 90])
def test_experts_block(n):
    blk = Block(n, 512, 768, 6, 2, 1)
    note("experts block n=%d" % n)
    x, y = (to_dev(synth.random_activations(s, n, 512)) for s in (1, 2))
    o = blk.run(x, y)
    torch.cuda.synchronize()
    blk.check(o)


def test_experts_block_in_a_graph():
    n = 40
    blk = Block(n, 512, 768, 6, 2, 2)
    x, y = (to_dev(synth.random_activations(s, n, 512)) for s in (3, 4))
    blk.run(x, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = blk.run(x, y)
    for s in (5, 6, 7):
        x.copy_(to_dev(synth.random_activations(s, n, 512)))
        note("experts block replay %d" % s)
        g.replay()
        torch.cuda.synchronize()
        e = blk.run(x, y)
        torch.cuda.synchronize()
        for key in ("r", "gate", "down", "out"):
            assert torch.equal(o[key], e[key]), key
        blk.check(o)


def test_route_more_ids_than_registers_hold():
    """70000 x 1 and 9000 x 8 ids: over 65536, where the sort reads its ids
    twice; checked against numpy's stable sort."""
    for n, experts, top in ((70001, 3, 1), (9001, 40, 8)):
        rng = np.random.default_rng([996, n])
        logits = rng.standard_normal((n, experts)).astype(np.float32)
        logits[rng.random(n) < 0.1] = -np.inf
        note("route n=%d experts=%d top=%d" % (n, experts, top))
        r = binding.route(to_dev(logits), top)
        torch.cuda.synchronize()
        order = np.argsort(-logits, axis=1, kind="stable")[:, :top].astype(np.int32)
        ids = np.where(np.take_along_axis(logits, order, 1) > -np.inf, order, -1)
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        flat = ids.reshape(-1)
        by = np.argsort(np.where(flat < 0, experts, flat), kind="stable")
        used = int((flat >= 0).sum())
        slot = np.full(flat.size, -1, np.int32)
        slot[by[:used]] = np.arange(used)
        assert np.array_equal(r.slot.cpu().numpy().reshape(-1), slot)
        rows = r.rows.cpu().numpy()
        assert np.array_equal(rows[:used], by[:used] // top) and (rows[used:] == -1).all()
        assert np.array_equal(r.offsets.cpu().numpy(), np.searchsorted(np.sort(flat[flat >= 0]), np.arange(experts + 1)))
