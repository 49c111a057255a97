"""The operators at sizes where a 32-bit offset would wrap: weights past 4 GiB,
outputs, inputs and activations of more than 2^31 values.  Inputs repeat a
small pool of rows, so that every row of a result has its counterpart in a
small call that the other tests hold to the definition."""
import numpy as np
import pytest
import torch

import operator_refs as refs
import oracle
from gpu_helpers import check_fp32, note, to_dev
from q4_q8_integer_amd import binding, synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _same_rows(big, small, index, what):
    """big[i] == small[index[i]] bit for bit, in pieces of 2^16 rows."""
    for a in range(0, big.shape[0], 1 << 16):
        part = big[a:a + (1 << 16)]
        assert torch.equal(part, small[index[a:a + part.shape[0]]]), "%s: rows from %d" % (what, a)


@pytest.mark.parametrize("fmt,block", [("q4k", 144), ("q6k", 210)])
@pytest.mark.parametrize("count", [3, 30, 200])
def test_grouped_weights_past_4_gib(fmt, block, count):
    """The last of 400 experts starts past 2^32 bytes; the first has slots too."""
    m, k, experts = 1288, 16384, 400
    note("large grouped weights %s count=%d" % (fmt, count))
    each = m * (k // 256) * block
    assert each * (experts - 1) > 2 ** 32
    w = [refs.weights(fmt, 50 + i, m, k) for i in range(2)]
    dw = torch.zeros(each * experts, dtype=torch.uint8, device=DEV)
    dw[:each] = to_dev(w[0].reshape(-1))
    dw[-each:] = to_dev(w[1].reshape(-1))
    rng = np.random.default_rng(count)
    q, ds = oracle.quantize(synth.random_activations(3, 8, k, "outliers"))
    rows = rng.integers(0, 8, 2 + count).astype(np.int32)
    off = np.full(experts + 1, 2, np.int32)
    off[0], off[-1] = 0, 2 + count
    out = binding.fold_grouped(binding.FORMAT_Q4K if fmt == "q4k" else binding.FORMAT_Q6K, dw, experts, m, k, to_dev(q),
                               to_dev(ds.view(np.int32)), to_dev(off), to_dev(rows))
    torch.cuda.synchronize()
    ref = [refs.fold64(fmt, x, m, k, q, ds) for x in w]
    check_fp32(out.cpu().numpy(), np.concatenate([ref[0][rows[:2]], ref[1][rows[2:]]]), "past 4 GiB")


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
def test_grouped_output_past_2_31_values(fmt):
    m, k, slots, pool = 2056, 256, (1 << 20) + 75, 64
    note("large grouped output %s" % fmt)
    w = [refs.weights(fmt, 60 + i, m, k) for i in range(2)]
    dw = to_dev(np.concatenate([x.reshape(-1) for x in w]))
    q, ds = oracle.quantize(synth.random_activations(4, pool, k, "outliers"))
    dq, dds = to_dev(q), to_dev(ds.view(np.int32))
    rows = torch.randint(0, pool, (slots,), dtype=torch.int32, device=DEV)
    cut = slots - 300
    f = binding.FORMAT_Q4K if fmt == "q4k" else binding.FORMAT_Q6K
    out = binding.fold_grouped(f, dw, 2, m, k, dq, dds, to_dev(np.array([0, cut, slots], np.int32)), rows)
    # each pool row 300 times over: the same kernel on few slots
    small = []
    for e in range(2):
        idx = torch.arange(pool, dtype=torch.int32, device=DEV).repeat(5)
        off = [0, pool * 5, pool * 5] if e == 0 else [0, 0, pool * 5]
        small.append(binding.fold_grouped(f, dw, 2, m, k, dq, dds, to_dev(np.array(off, np.int32)), idx)[:pool].clone())
    torch.cuda.synchronize()
    for e in range(2):
        check_fp32(small[e].cpu().numpy(), refs.fold64(fmt, w[e], m, k, q, ds), "pool")
    _same_rows(out[:cut], small[0], rows[:cut].long(), "first expert")
    _same_rows(out[cut:], small[1], rows[cut:].long(), "second expert")


def test_epilogue_output_past_2_31_values():
    m, k, n, pool = 2056, 256, (1 << 20) + 75, 256
    note("large epilogue output")
    w = to_dev(refs.weights("q4k", 70, m, k).reshape(-1))
    q, ds = oracle.quantize(synth.random_activations(5, pool, k, "outliers"))
    idx = torch.randint(0, pool, (n,), device=DEV)
    dq, dds = to_dev(q), to_dev(ds.view(np.int32))
    bias = torch.randn(m, device=DEV)
    call = lambda a, b: binding.fold_epilogue(binding.FORMAT_Q4K, w, m, k, a, b, bias, binding.ACT_SILU)
    out, small = call(dq[idx].contiguous(), dds[idx].contiguous()), call(dq, dds)
    torch.cuda.synchronize()
    _same_rows(out, small, idx, "epilogue")


def test_epilogue_q6k_past_4_gib_of_codes():
    """A small matrix on so many long rows that their codes pass 4 GiB: the
    binary16 kernel, with the fold entry point's bits."""
    m, k, n, pool = 16, 65792, 65536, 64
    assert n * k > 2 ** 32
    note("large q6_K epilogue")
    w = to_dev(refs.weights("q6k", 71, m, k).reshape(-1))
    q, ds = oracle.quantize(synth.random_activations(6, pool, k, "outliers"))
    idx = torch.randint(0, pool, (n,), device=DEV)
    dq, dds = to_dev(q)[idx].contiguous(), to_dev(ds.view(np.int32))[idx].contiguous()
    out, fold = binding.fold_epilogue(binding.FORMAT_Q6K, w, m, k, dq, dds), binding.q6k_fp32(w, m, k, dq, dds)
    torch.cuda.synchronize()
    assert torch.equal(out, fold)
    check_fp32(out[-200:].cpu().numpy(), refs.fold64("q6k", w.cpu().numpy().reshape(m, -1), m, k, q, ds)[idx[-200:].cpu()],
               "last rows")


def test_norm_past_2_31_values():
    k, n, pool = 4128, (1 << 19) + 3, 64
    assert n * k > 2 ** 31
    note("large norm")
    base, y = torch.randn(pool, k, device=DEV), torch.randn(pool, k, device=DEV).half()
    weight = 1 + 0.1 * torch.randn(k, device=DEV)
    idx = torch.arange(n, device=DEV) % pool
    q, ds, r = binding.quantize_norm(base[idx], weight, y=y[idx], residual_scale=0.5)
    sq, sds, sr = binding.quantize_norm(base, weight, y=y, residual_scale=0.5)
    torch.cuda.synchronize()
    _same_rows(r, sr, idx, "r")
    _same_rows(q, sq, idx, "q")
    _same_rows(ds, sds, idx, "ds")


def test_combine_past_2_31_values():
    m, n = 2056, (1 << 20) + 75
    note("large combine")
    y = torch.randn(n, m, device=DEV).half()
    slot = torch.randperm(n, device=DEV).int()[:, None].contiguous()
    weight = torch.rand(n, 1, device=DEV)
    out = binding.combine(y, slot, weight)
    torch.cuda.synchronize()
    for a in range(0, n, 1 << 16):   # one expert: a single product, rounded once
        part = slice(a, a + (1 << 16))
        assert torch.equal(out[part], weight[part] * y[slot[part, 0].long()].float()), a


@pytest.mark.parametrize("fmt", ["q4k", "q6k"])
def test_grouped_output_of_2_35_values(fmt):
    """Where one slot per item and 16 rows per tile would be more than 2^31
    tiles (the kernels' items are larger)."""
    m, k, slots, pool = 16384, 256, 1 << 21, 64
    note("large grouped output, 2^35 values, %s" % fmt)
    w = [refs.weights(fmt, 62 + i, m, k) for i in range(2)]
    dw = to_dev(np.concatenate([x.reshape(-1) for x in w]))
    q, ds = oracle.quantize(synth.random_activations(4, pool, k, "outliers"))
    dq, dds = to_dev(q), to_dev(ds.view(np.int32))
    rows = torch.randint(0, pool, (slots,), dtype=torch.int32, device=DEV)
    cut = slots - 300
    f = binding.FORMAT_Q4K if fmt == "q4k" else binding.FORMAT_Q6K
    out = binding.fold_grouped(f, dw, 2, m, k, dq, dds, to_dev(np.array([0, cut, slots], np.int32)), rows, f16=True)
    idx = torch.arange(pool, dtype=torch.int32, device=DEV).repeat(5)
    for e, (a, b) in enumerate(((0, cut), (cut, slots))):
        off = [0, pool * 5, pool * 5] if e == 0 else [0, 0, pool * 5]
        small = binding.fold_grouped(f, dw, 2, m, k, dq, dds, to_dev(np.array(off, np.int32)), idx)[:pool].clone()
        torch.cuda.synchronize()
        check_fp32(small.cpu().numpy(), refs.fold64(fmt, w[e], m, k, q, ds), "pool")
        _same_rows(out[a:b], small.half(), rows[a:b].long(), "expert %d" % e)


@pytest.mark.parametrize("f16,m", [(True, 2 ** 31 - 1), (True, 2 ** 31 - 8), (False, 2 ** 31 - 4)])
def test_combine_columns_up_to_the_last_int(f16, m):
    """Rows of nearly 2^31 columns, where m and a workgroup's columns together
    pass an int: by value and by 16 bytes."""
    note("combine m=%d" % m)
    y = (torch.arange(m, device=DEV, dtype=torch.int32) % 2039).to(torch.float16 if f16 else torch.float32)[None, :]
    out = torch.full((1, m), 7.0, device=DEV)
    got = binding.combine(y, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.full((1, 1), 0.5, device=DEV),
                          out=out)
    torch.cuda.synchronize()
    assert got is out
    for a in range(0, m, 1 << 28):
        part = slice(a, min(a + (1 << 28), m))
        assert torch.equal(out[0, part], 0.5 * y[0, part].float()), a


def test_combine_of_2_32_values():
    m, n, slots = 4096, (1 << 20) + 3, 70
    note("combine n=%d m=%d" % (n, m))
    y = torch.randn(slots, m, device=DEV).half()
    slot = torch.randint(0, slots, (n, 1), dtype=torch.int32, device=DEV)
    weight = torch.rand(n, 1, device=DEV)
    out = binding.combine(y, slot, weight)
    torch.cuda.synchronize()
    for a in range(0, n, 1 << 16):   # one expert: a single product, rounded once
        part = slice(a, a + (1 << 16))
        assert torch.equal(out[part], weight[part] * y[slot[part, 0].long()].float()), a


def test_route_of_the_most_tokens():
    """2^26 - 4 tokens, the launch's limit, two experts."""
    n = (1 << 26) - 4
    note("route n=%d" % n)
    logits = torch.randn(n, 2, device=DEV)
    logits[::9] = -float("inf")
    r = binding.route(logits, 1)
    live, second = logits[:, 0] > -float("inf"), logits[:, 1] > logits[:, 0]
    torch.cuda.synchronize()
    ids = torch.where(live, second.int(), -1)
    assert torch.equal(r.ids[:, 0], ids)
    assert torch.equal(r.weights[:, 0], live.float())
    first, used = int((ids == 0).sum()), int(live.sum())
    assert r.offsets.tolist() == [0, first, used]
    rows = torch.cat([(ids == e).nonzero()[:, 0] for e in (0, 1)]).int()
    assert torch.equal(r.rows[:used], rows) and (r.rows[used:] == -1).all()
    slot = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    slot[rows.long()] = torch.arange(used, dtype=torch.int32, device=DEV)
    assert torch.equal(r.slot[:, 0], slot)
