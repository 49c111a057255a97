"""mmq_fold_grouped on the GPU against the 64-bit fold of each expert: ragged
groups on both sides of every kernel border, empty experts, many experts,
gathered rows, epilogues, slots outside the groups, wrong offsets and rows,
streams and graphs."""
import numpy as np
import pytest
import torch

import operator_refs as refs
import oracle
from gpu_helpers import check_fp32, note, to_dev
from q4_q8_integer_amd import binding, synth

pytestmark = pytest.mark.gpu
FMT = {"q4k": binding.FORMAT_Q4K, "q6k": binding.FORMAT_Q6K}


class Case:
    def __init__(self, fmt, counts, m, k, seed=0, first=0, tail=0, tokens=None):
        rng = np.random.default_rng([990, seed, m, k, len(counts)])
        self.fmt, self.counts, self.m, self.k, self.experts = fmt, counts, m, k, len(counts)
        self.offsets = (first + np.concatenate(([0], np.cumsum(counts)))).astype(np.int32)
        self.slots = int(self.offsets[-1]) + tail
        self.w = [refs.weights(fmt, 10 * seed + e, m, k) for e in range(self.experts)]
        self.tokens = tokens or max(self.slots, 1)
        x = synth.random_activations(seed, self.tokens, k, "outliers")
        self.q, self.ds = oracle.quantize(x)
        self.rows = rng.integers(0, tokens, self.slots).astype(np.int32) if tokens else None
        self.dw = to_dev(np.concatenate([w.reshape(-1) for w in self.w]))
        self.dq, self.dds = to_dev(self.q), to_dev(self.ds.view(np.int32))
        self.doff = to_dev(self.offsets)
        self.drows = None if self.rows is None else to_dev(self.rows)

    def fold(self):
        """float64 [slots, m]; rows outside the groups NaN."""
        out = np.full((self.slots, self.m), np.nan)
        for e in range(self.experts):
            a, b = self.offsets[e], self.offsets[e + 1]
            if a < b:
                at = np.arange(a, b) if self.rows is None else self.rows[a:b]
                out[a:b] = refs.fold64(self.fmt, self.w[e], self.m, self.k, self.q[at], self.ds[at])
        return out

    def call(self, **kw):
        return binding.fold_grouped(FMT[self.fmt], self.dw, self.experts, self.m, self.k, self.dq, self.dds, self.doff,
                                    self.drows, **kw)

    def check(self, what, f16=False):
        note("grouped %s: %s m=%d k=%d counts=%s" % (what, self.fmt, self.m, self.k, list(self.counts)[:12]))
        out = torch.full((self.slots, self.m), 77.0, device="cuda:0", dtype=torch.float16 if f16 else torch.float32)
        got = self.call(out=out, f16=f16)
        torch.cuda.synchronize()
        assert got is out
        got, ref = got.cpu().numpy(), self.fold()
        used = ~np.isnan(ref[:, 0])
        assert (got[~used] == 77).all(), "rows outside the groups are left as they were"
        if f16:
            bound = refs.U16 * np.abs(ref[used]) * (1 + 1e-3) + 1e-3 * np.abs(ref[used]).max(1, keepdims=True) + refs.SUB16
            assert (np.abs(got[used].astype(np.float64) - ref[used]) <= bound).all()
        elif used.any():
            check_fp32(got[used], ref[used], what)
        return got


BORDERS = [0, 1, 4, 5, 0, 8, 9, 16, 17, 3, 63, 64, 65, 0, 128, 129, 2, 200]


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_borders(fmt, gather):
    """Group sizes around 4, 8 and 16 slots (few-token items), 8 and 16 (kernel
    borders), 64 and 128 (tiles), with empty experts between them."""
    Case(fmt, BORDERS, 136, 512, 1, first=3, tail=5, tokens=50 if gather else None).check("borders")


@pytest.mark.parametrize("fmt,m,k", [("q4k", 1, 256), ("q4k", 131, 768), ("q4k", 300, 2304), ("q6k", 8, 256),
                                     ("q6k", 136, 768), ("q6k", 264, 2304), ("q4k", 8192, 8192), ("q6k", 16, 16640)])
def test_grouped_shapes(fmt, m, k):
    Case(fmt, [2, 0, 7, 33, 1], m, k, 2, tokens=5).check("shapes")


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("counts", [[1], [3], [0, 2], [1, 0, 0, 1, 1], [4], [16], [17], [40, 0], [300], [1] * 9, [6] * 5],
                         ids=str)
def test_grouped_small_calls(fmt, counts):
    Case(fmt, counts, 72, 512, 3).check("small")


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("counts", [[5, 0, 16, 1], [31, 17, 2, 64, 16, 49]], ids=["mean below 16", "mean above 16"])
@pytest.mark.parametrize("m,k", [(24, 256 * 5), (264, 256 * 17), (2056, 768), (24584, 256)])
def test_grouped_few_forms(fmt, counts, m, k):
    """Both forms of the few-token kernel, from units whose k eight waves share
    to workgroups that go over many units with a wave per row tile."""
    Case(fmt, counts, m, k, 20, tokens=33).check("few forms")


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("count", [3, 20])
def test_grouped_few_long_rows(fmt, count):
    """More than 256 super-blocks per wave, where the sums move on."""
    Case(fmt, [count], 24, 256 * 2100, 21, tokens=4).check("long rows")


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("experts", [63, 64, 65, 130])
def test_grouped_many_experts(fmt, experts):
    """More experts than a wave has lanes: items are found across the scans."""
    rng = np.random.default_rng(experts)
    counts = rng.integers(0, 4, experts)
    counts[rng.integers(0, experts, 3)] = [20, 70, 9]
    counts[-1] = 18
    Case(fmt, counts.tolist(), 40, 256, 4, tokens=30).check("many")


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
def test_grouped_all_empty_and_no_slots(fmt):
    c = Case(fmt, [0, 0, 0], 32, 256, 5, first=2, tail=6)
    c.check("empty")
    c.doff = torch.zeros(4, dtype=torch.int32, device="cuda:0")
    out = c.call(out=torch.empty((0, 32), device="cuda:0"))
    assert out.shape == (0, 32)


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("act", [binding.ACT_NONE, binding.ACT_SILU, binding.ACT_GELU_TANH])
def test_grouped_epilogue(fmt, f16, act):
    """Bias rows per expert, activation and residual against the same call's
    plain float32 result."""
    for m in (64, 72 if fmt == "q6k" else 67):
        c = Case(fmt, [5, 0, 20, 70, 1, 16], m, 512, 6, first=1, tail=2, tokens=40)
        plain = c.check("epilogue base")
        rng = np.random.default_rng(m)
        b = rng.standard_normal((c.experts, m)).astype(np.float32)
        r = rng.standard_normal((c.slots, m)).astype(np.float16 if act else np.float32)
        got = c.call(bias=to_dev(b), activation=act, residual=to_dev(r), f16=f16)
        torch.cuda.synchronize()
        got = got.cpu().numpy()
        e = np.repeat(np.arange(c.experts), c.counts)
        a, z = c.offsets[0], c.offsets[-1]
        refs.check_epilogue(got[a:z], plain[a:z], b[e], act, r[a:z], f16, "grouped m=%d" % m)


def test_grouped_equals_the_fold_of_each_expert():
    """A group's float32 results are the fold entry point's on the kernel of
    the same tiling: above 64 tokens, bit for bit."""
    c = Case("q4k", [70, 0, 65], 256, 1024, 7)
    got = c.check("equal")
    for e, (a, b) in enumerate(zip(c.offsets[:-1], c.offsets[1:])):
        if a < b:
            ref = binding.fp32(to_dev(c.w[e].reshape(-1)), c.m, c.k, c.dq[a:b].contiguous(), c.dds[a:b].contiguous())
            torch.cuda.synchronize()
            assert np.array_equal(ref.cpu().numpy(), got[a:b])


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
def test_grouped_strided_output(fmt):
    c = Case(fmt, [3, 20, 0, 80], 40, 256, 8)
    plain = c.check("strided base")
    wide = torch.full((c.slots, 64), 3.0, device="cuda:0")
    c.call(out=wide[:, 8:48])
    torch.cuda.synchronize()
    assert (wide[:, :8] == 3).all() and (wide[:, 48:] == 3).all()
    assert np.array_equal(wide[:, 8:48].cpu().numpy(), plain)


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
def test_grouped_clamps_wrong_rows_and_offsets(fmt):
    """Offsets and rows out of range are clamped: the good groups are right
    and nothing around the output changes."""
    c = Case(fmt, [4, 30, 2], 40, 256, 9, tokens=12)
    ref = c.fold()
    n = c.slots
    c.drows = to_dev(np.where(np.arange(n) >= 4, [-5, 1 << 30][0], c.rows).astype(np.int32))
    buf = torch.full((n + 8, 40), 9.0, device="cuda:0")
    for off in ([0, 4, n + 1000, n], [0, 4, 2, 1], [-7, 4, 1 << 30, -1]):
        buf.fill_(9.0)
        c.doff = to_dev(np.array(off, np.int32))
        note("grouped clamped %s %s" % (fmt, off))
        c.call(out=buf[4:4 + n])
        torch.cuda.synchronize()
        assert (buf[:4] == 9).all() and (buf[4 + n:] == 9).all()
        check_fp32(buf[4:8].cpu().numpy(), ref[:4], "first group")


def test_grouped_graph_replays_over_new_offsets():
    """One captured call follows the offsets: replayed for groups of other
    sizes, with eager calls between."""
    c = Case("q4k", [5, 40, 0, 70, 13], 136, 512, 10)
    out = torch.zeros((c.slots, c.m), device="cuda:0")
    c.call(out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(out=out)
    n = c.slots
    for cuts in ([0, 1, 2, 100, n], [0, 0, 0, 0, n], [16, 33, 33, 97, n], [3, 20, 90, 90, 91]):
        c.doff.copy_(to_dev(np.array([0] + list(cuts), np.int32)))
        out.fill_(1.0)
        g.replay()
        eager = torch.full_like(out, 1.0)
        c.call(out=eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        c.offsets = c.doff.cpu().numpy()
        c.counts = np.diff(c.offsets).tolist()
        ref = c.fold()
        used = ~np.isnan(ref[:, 0])
        check_fp32(out.cpu().numpy()[used], ref[used], "replay")


def test_grouped_two_streams():
    a, b = (Case("q4k", [9, 33, 0, 80], 200, 512, s) for s in (11, 12))
    ra, rb = a.call(), b.call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(s):
            oa = a.call()
        ob = b.call()
        torch.cuda.synchronize()
        assert torch.equal(oa, ra) and torch.equal(ob, rb)


def test_grouped_binding_refusals():
    c = Case("q4k", [2, 3], 32, 256, 13, tokens=4)
    with pytest.raises(ValueError):
        c.call(bias=torch.zeros(32, device="cuda:0"))
    with pytest.raises(ValueError):
        binding.fold_grouped(binding.FORMAT_Q4K_TILES, c.dw, 2, 32, 256, c.dq, c.dds, c.doff)
    with pytest.raises(ValueError):
        binding.fold_grouped(binding.FORMAT_Q4K, c.dw, 3, 32, 256, c.dq, c.dds, c.doff)
    with pytest.raises(TypeError):
        binding.fold_grouped(binding.FORMAT_Q4K, c.dw, 2, 32, 256, c.dq, c.dds, c.doff.long())
    with pytest.raises(ValueError):
        binding.fold_grouped(binding.FORMAT_Q4K, c.dw, 2, 32, 256, c.dq, c.dds, c.doff[:2].contiguous())
