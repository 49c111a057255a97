"""mmq_fold_grouped where its arguments are wrong or at a border: offsets that
decrease, rows out of range on both sides, groups at the kernels' borders, and
codes past 2^31 bytes."""
import numpy as np
import pytest
import torch

import operator_refs as refs
import oracle
from gpu_helpers import check_fp32, note, to_dev
from q4_q8_integer_amd import binding, synth

pytestmark = pytest.mark.gpu
FMT = {"q4k": binding.FORMAT_Q4K, "q6k": binding.FORMAT_Q6K}


class Problem:
    """experts matrices of m x k, and `tokens` rows of codes."""

    def __init__(self, fmt, experts, m, k, tokens, seed):
        self.fmt, self.experts, self.m, self.k = fmt, experts, m, k
        self.w = [refs.weights(fmt, 700 + 10 * seed + e, m, k) for e in range(experts)]
        self.q, self.ds = oracle.quantize(synth.random_activations(seed, tokens, k, "outliers"))
        self.dw = to_dev(np.concatenate([w.reshape(-1) for w in self.w]))
        self.dq, self.dds = to_dev(self.q), to_dev(self.ds.view(np.int32))

    def fold(self, e, rows):
        return refs.fold64(self.fmt, self.w[e], self.m, self.k, self.q[rows], self.ds[rows])

    def call(self, offsets, rows, **kw):
        return binding.fold_grouped(FMT[self.fmt], self.dw, self.experts, self.m, self.k, self.dq, self.dds,
                                    to_dev(np.array(offsets, np.int32)), to_dev(np.asarray(rows, np.int32)), **kw)


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("n", [10, 30, 200])
def test_decreasing_offsets_leave_the_groups_apart(fmt, n):
    """An offset below an earlier one counts as the largest before it, over the
    64 experts that a wave looks at together and beyond: no slot belongs to two
    experts (which would write it in no fixed order, and go over every item
    once for each of them)."""
    p = Problem(fmt, 3, 40, 256, 20, 1)
    rows = np.random.default_rng(n).integers(0, 20, n)
    for off, groups in (([0, n, 0, n], {0: (0, n)}), ([0, n // 2, 1, n], {0: (0, n // 2), 2: (n // 2, n)}),
                        ([n // 3, 0, n, 5], {1: (n // 3, n)}), ([-9, 4, 2, n + 77], {0: (0, 4), 2: (4, n)})):
        note("grouped decreasing %s %s" % (fmt, off))
        out = torch.full((n, p.m), 9.0, device="cuda:0")
        p.call(off, rows, out=out)
        torch.cuda.synchronize()
        out = out.cpu().numpy()
        left = np.ones(n, bool)
        for e, (a, b) in groups.items():
            check_fp32(out[a:b], p.fold(e, rows[a:b]), "expert %d of %s" % (e, off))
            left[a:b] = False
        assert (out[left] == 9).all()


@pytest.mark.parametrize("n", [10, 200])
def test_decreasing_offsets_of_many_experts(n):
    p = Problem("q4k", 131, 8, 256, 5, 2)
    rows = np.random.default_rng(n).integers(0, 5, n)
    off = np.zeros(132, np.int32)
    off[64:] = n - 1                    # the first 64 experts have none, the next one all but a slot
    off[65:130:2] = 3                   # and then they go down and up
    off[131] = n
    note("grouped decreasing, 131 experts")
    out = torch.full((n, p.m), 9.0, device="cuda:0")
    p.call(off, rows, out=out)
    torch.cuda.synchronize()
    out = out.cpu().numpy()
    check_fp32(out[:n - 1], p.fold(63, rows[:n - 1]), "expert 63")
    check_fp32(out[n - 1:], p.fold(130, rows[n - 1:]), "the last expert")


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("n", [9, 30, 200])
def test_rows_out_of_range_on_both_sides(fmt, n):
    """Rows below 0 count as the first row of q, rows past its end as the last,
    in every kernel's range."""
    p = Problem(fmt, 2, 40, 512, 12, 3)
    rows = np.random.default_rng(n).integers(0, 12, n + 5)
    bad = np.array([-5, 1 << 30, 12, -1, -(1 << 31), (1 << 31) - 1])
    rows[2:n:2] = bad[np.arange(len(rows[2:n:2])) % 6]
    note("grouped rows out of range %s n=%d" % (fmt, n))
    out = p.call([0, n, n + 5], rows)
    torch.cuda.synchronize()
    at = np.clip(rows, 0, 11)
    check_fp32(out[:n].cpu().numpy(), p.fold(0, at[:n]), "clamped")
    check_fp32(out[n:].cpu().numpy(), p.fold(1, at[n:]), "in range")


# The kernels' borders: 16 slots (one token tile), 32 (q4_K) and 64 (q6_K), 64
# and 128 (binary16 items), with the mean below 16 slots, where the one-tile
# form is launched, and above.
@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("counts", [[15, 0, 31], [16, 32, 0, 0, 0, 0], [17, 33, 0, 0, 0, 0], [31, 32, 33], [16, 17, 15, 32],
                                    [32], [33], [63, 64, 65], [64, 0, 0, 0, 0, 0], [65, 0, 0, 0, 0, 0], [127, 128, 129],
                                    [95, 97], [32, 33, 64, 65, 1, 16, 17, 2, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0]], ids=str)
def test_groups_at_the_kernels_borders(fmt, counts):
    p = Problem(fmt, len(counts), 72, 768, 50, 4)
    rows = np.random.default_rng(sum(counts)).integers(0, 50, sum(counts))
    off = np.concatenate(([0], np.cumsum(counts)))
    note("grouped borders %s %s" % (fmt, counts))
    out = p.call(off, rows)
    torch.cuda.synchronize()
    out = out.cpu().numpy()
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if a < b:
            check_fp32(out[a:b], p.fold(e, rows[a:b]), "expert %d" % e)


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
def test_rows_of_codes_past_2_31_bytes(fmt):
    """Gathered rows on both sides of 2^31 bytes of codes and up to the 2^32
    that are allowed, where byte offsets pass an int; in each kernel."""
    m, k, pool = 24, 4096, 64
    tokens = (1 << 20) - 1
    assert 1 << 31 < tokens * k < 1 << 32
    note("grouped codes past 2^31 bytes %s" % fmt)
    p = Problem(fmt, 3, m, k, pool, 5)
    p.dq = p.dq.repeat((tokens + pool - 1) // pool, 1)[:tokens].contiguous()
    p.dds = p.dds.repeat((tokens + pool - 1) // pool, 1)[:tokens].contiguous()
    counts = [12, 30, 200]
    rng = np.random.default_rng(7)
    rows = rng.integers(tokens // 2 - 3, tokens, sum(counts))
    rows[[0, 12, 42]], rows[[1, 13, 43]] = tokens - 1, (1 << 19) - 1
    off = np.concatenate(([0], np.cumsum(counts)))
    out = p.call(off, rows)
    torch.cuda.synchronize()
    for e in range(3):
        a, b = off[e], off[e + 1]
        check_fp32(out[a:b].cpu().numpy(), p.fold(e, rows[a:b] % pool), "expert %d" % e)


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("m,pad", [(72, 0), (72, 8), (40, 3)])
def test_residual_in_place(fmt, f16, m, pad):
    """x += the experts' products, in the output's own rows (of a wider array
    too), in every kernel: each value is read and written once, and rows
    outside the groups and columns beside them keep theirs."""
    counts = [9, 30, 0, 70, 150]
    p = Problem(fmt, len(counts), m, 512, 30, 6)
    n = sum(counts) + 7
    rng = np.random.default_rng([m, pad, f16])
    rows = rng.integers(0, 30, n)
    off = 4 + np.concatenate(([0], np.cumsum(counts)))
    dt = torch.float16 if f16 else torch.float32
    note("grouped in place %s f16=%s m=%d pad=%d" % (fmt, f16, m, pad))
    used = slice(off[0], off[-1])
    plain = p.call(off, rows)[used].cpu().numpy()
    x = rng.standard_normal((n, m + pad)).astype(np.float16 if f16 else np.float32)
    buf = to_dev(x)
    out = buf[:, :m]
    assert p.call(off, rows, residual=out, out=out, f16=f16) is out
    torch.cuda.synchronize()
    got = buf.cpu().numpy()
    assert np.array_equal(got[:, m:], x[:, m:])
    assert np.array_equal(got[:off[0]], x[:off[0]]) and np.array_equal(got[off[-1]:], x[off[-1]:])
    refs.check_epilogue(got[used, :m], plain, None, 0, x[used, :m], f16, "in place")
