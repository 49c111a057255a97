"""The epilogue's activations on exact float32 values, in both tails: weights
of zero bytes make every fold 0, so that the value is the bias."""
import numpy as np
import pytest
import torch

import activation_bounds as ab
import operator_refs as refs
from gpu_helpers import note, to_dev
from q4_q8_integer_amd import binding, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("fmt,n", [(binding.FORMAT_Q4K, 1), (binding.FORMAT_Q4K, 100), (binding.FORMAT_Q6K, 20)])
def test_activations_of_exact_values(act, fmt, n):
    v = ab.values(act)
    m, k = v.size, 256
    block = 210 if fmt == binding.FORMAT_Q6K else 144
    w = torch.zeros(m * block, dtype=torch.uint8, device="cuda:0")
    q, ds = binding.quantize(to_dev(synth.random_activations(1, n, k)))
    note("activations act=%d fmt=%d n=%d" % (act, fmt, n))
    out = binding.fold_epilogue(fmt, w, m, k, q, ds, to_dev(v), act)
    half = binding.fold_epilogue(fmt, w, m, k, q, ds, to_dev(v), act, f16=True)
    torch.cuda.synchronize()
    out = out.cpu().numpy()
    for row in (out[0], out[-1]):
        bad = ab.off(row, v, act)
        ref = refs.act64(v.astype(np.float64), act)
        units = np.abs(row - ref) / np.maximum(np.abs(ref) * ab.U, 1e-300)
        assert not bad.any(), "act %d: %d off, first at v = %r (%r for %r, %.1f half steps)" % (
            act, bad.sum(), v[bad][0], row[bad][0], ref[bad][0], units[bad][0])
    with np.errstate(over="ignore"):
        assert np.array_equal(half.cpu().numpy(), out.astype(np.float16))   # rounded once, from the float32 value
