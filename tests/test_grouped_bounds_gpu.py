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
