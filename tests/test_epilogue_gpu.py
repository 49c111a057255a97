"""mmq_fold_epilogue on the GPU: bit for bit the fold entry point without
operands, and the 64-bit epilogue of its float32 result with them, over every
format, every kernel the automatic choice takes, and every operand."""
import numpy as np
import pytest
import torch

import operator_refs as refs
from gpu_helpers import check_fp32, host_ds, note, to_dev
from q4_q8_integer_amd import binding, synth

pytestmark = pytest.mark.gpu

FORMATS = {"q4k": (binding.FORMAT_Q4K, binding.FORMAT_Q4K_REPACKED, binding.FORMAT_Q4K_TILES,
                   binding.FORMAT_Q4K_REPACKED_TILES),
           "q6k": (binding.FORMAT_Q6K, binding.FORMAT_Q6K_TILES)}


def _plain(fmt, w, m, k, q, ds):
    if fmt == binding.FORMAT_Q4K:
        return binding.fp32(w, m, k, q, ds)
    if fmt == binding.FORMAT_Q4K_REPACKED:
        return binding.fp32_repacked(w, m, k, q, ds)
    if fmt == binding.FORMAT_Q6K:
        return binding.q6k_fp32(w, m, k, q, ds)
    if fmt == binding.FORMAT_Q6K_TILES:
        return binding.q6k_fp32_tiles(w, m, k, q, ds)
    return binding.fp32_tiles(w, m, k, q, ds, repacked=fmt == binding.FORMAT_Q4K_REPACKED_TILES)


def _setup(fmt, seed, m, k, n):
    base = "q6k" if fmt in FORMATS["q6k"] else "q4k"
    w = to_dev(refs.weights(base, seed, m, k).reshape(-1))
    if fmt in (binding.FORMAT_Q4K_REPACKED, binding.FORMAT_Q4K_REPACKED_TILES):
        w = binding.repack(w, m, k)
    x = to_dev(synth.random_activations(seed, n, k) / np.float32(np.sqrt(k)))
    q, ds = binding.quantize_tiled(x) if fmt in binding._TILE_FORMATS else binding.quantize(x)
    return w, q, ds


def _own(fmt, m, n):
    """Whether the call runs a kernel that the fold entry point does not."""
    return fmt == binding.FORMAT_Q6K and n > 8 and (n <= 64 or -(-m // 16) * -(-n // 64) <= 1536)


def _case(fmt, m, k, n, act, residual, f16, bias=True, seed=0):
    note("epilogue fmt=%d m=%d k=%d n=%d act=%d residual=%s f16=%s" % (fmt, m, k, n, act, residual, f16))
    w, q, ds = _setup(fmt, seed + n, m, k, n)
    rng = np.random.default_rng([980, seed, m, n])
    b = rng.standard_normal(m).astype(np.float32) if bias else None
    r = None if residual is None else rng.standard_normal((n, m)).astype(residual)
    fold = _plain(fmt, w, m, k, q, ds)
    same = binding.fold_epilogue(fmt, w, m, k, q, ds, f16=f16)
    out = binding.fold_epilogue(fmt, w, m, k, q, ds, None if b is None else to_dev(b), act,
                                None if r is None else to_dev(r), f16=f16)
    torch.cuda.synchronize()
    if _own(fmt, m, n):
        # a kernel of its own: its fold is held to the oracle, and the epilogue to its fold
        fold = binding.fold_epilogue(fmt, w, m, k, q, ds)
        torch.cuda.synchronize()
        check_fp32(fold.cpu().numpy(), refs.fold64("q6k", w.cpu().numpy().reshape(m, -1), m, k, q.cpu().numpy(),
                                                   host_ds(ds)), "q6k few")
    assert torch.equal(same, fold.half() if f16 else fold), "without operands the call is the fold"
    refs.check_epilogue(out.cpu().numpy(), fold.cpu().numpy(), b, act, r, f16,
                        "fmt %d m %d k %d n %d act %d" % (fmt, m, k, n, act))


# Token counts on both sides of every kernel border of a small matrix: narrow
# (1-16), few-token (17-64), binary16; dot4 of q6_K (1-8); slices of 8 tokens
# of the repacked dot4 kernel.
@pytest.mark.parametrize("n", [1, 5, 8, 12, 17, 33, 50, 65, 130])
@pytest.mark.parametrize("fmt", range(6))
def test_epilogue_formats_and_kernels(fmt, n):
    act = (fmt + n) % 5
    m = 131 if n % 2 else 132                # odd rows: no 16-byte stores
    _case(fmt, m, 512, n, act, [None, np.float32, np.float16][(fmt + n) % 3], (fmt * 3 + n) % 2 == 0)


@pytest.mark.parametrize("n", [9, 16, 17, 31, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("m,k", [(1, 256), (37, 2048), (130, 2304), (48, 16640)])
def test_q6k_few_tokens(m, k, n):
    """Every token-tile count of the q6_K few-token kernel: row tiles that end
    inside 16 rows and inside a 16-byte piece, one super-block (seven idle
    waves), a whole round of the waves, one more, and 65."""
    _case(binding.FORMAT_Q6K, m, k, n, n % 5, np.float32, n % 2 == 0, seed=11)


@pytest.mark.parametrize("n", [65, 128, 129, 200, 300])
@pytest.mark.parametrize("m,k", [(1, 256), (37, 2048), (260, 4352), (1030, 768)])
def test_q6k_more_tokens_on_small_matrices(m, k, n):
    """Above 64 tokens the streaming kernel takes several items of 64."""
    assert _own(binding.FORMAT_Q6K, m, n)
    _case(binding.FORMAT_Q6K, m, k, n, n % 5, np.float16 if m % 4 else np.float32, n % 2 == 0, seed=14)


@pytest.mark.parametrize("act", [0, 2, 3])
@pytest.mark.parametrize("m,n", [(16404, 129), (33000, 65), (16401, 130)])
def test_q6k_binary16_kernel(m, n, act):
    """Enough tiles for the binary16 kernel: the fold entry point's bits."""
    assert not _own(binding.FORMAT_Q6K, m, n)
    _case(binding.FORMAT_Q6K, m, 512, n, act, np.float32, act == 2, seed=15)


@pytest.mark.parametrize("n", [9, 16, 17, 33, 64])
@pytest.mark.parametrize("m,k", [(4097, 256), (4120, 4352), (8200, 768), (12300, 512)])
def test_q6k_few_tokens_tall(m, k, n):
    """Above 4096 rows, where the streaming kernel runs: one to 16 waves on a
    row tile, and workgroups that go over several units."""
    _case(binding.FORMAT_Q6K, m, k, n, n % 5, np.float32, n % 2 == 0, seed=13)


def test_q6k_few_tokens_long_rows():
    """Beyond 32 super-blocks per wave, where the sums move on."""
    _case(binding.FORMAT_Q6K, 20, 256 * 600, 20, 0, None, False, bias=False, seed=12)


# Shapes that reach the dot4 (1 token), stream (3, 7, 12) and few-token (12 on
# 5001 rows) kernels of q4_K.
@pytest.mark.parametrize("m,k,n,kernel", [(14337, 4096, 1, binding.KERNEL_DOT4), (14337, 4096, 3, binding.KERNEL_STREAM),
                                          (14337, 4096, 7, binding.KERNEL_STREAM), (20000, 5120, 2, binding.KERNEL_NARROW),
                                          (5001, 256, 12, binding.KERNEL_FEW), (16384, 1024, 6, binding.KERNEL_NARROW)])
def test_epilogue_tall_matrices(m, k, n, kernel):
    assert binding.mmq_kernel_choice(binding.FORMAT_Q4K, m, k, n) == kernel
    _case(binding.FORMAT_Q4K, m, k, n, binding.ACT_SILU, np.float32, False, seed=3)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("f16", [False, True])
def test_activations_over_their_range(act, f16):
    """A bias from -130 to 130 over a small fold: both tails, and zero."""
    m, k, n = 1024, 256, 3
    w, q, ds = _setup(binding.FORMAT_Q4K, 5, m, k, n)
    fold = binding.fp32(w, m, k, q, ds)
    b = np.linspace(-130, 130, m).astype(np.float32)
    b[::97] = 0
    if act == binding.ACT_GELU:
        # beyond |v| = 13.5 the exact value leaves float32's normal range
        b = (b / 10).astype(np.float32)
    out = binding.fold_epilogue(binding.FORMAT_Q4K, w, m, k, q, ds, to_dev(b), act, f16=f16)
    torch.cuda.synchronize()
    refs.check_epilogue(out.cpu().numpy(), fold.cpu().numpy(), b, act, None, f16, "act %d" % act)


def test_lowest_bias_and_far_tails_are_finite():
    """Biases at the type's lowest and highest values (a masked output): no
    NaN, and the tails are 0 or the value itself."""
    m, k, n = 64, 256, 2
    w, q, ds = _setup(binding.FORMAT_Q4K, 6, m, k, n)
    low = torch.finfo(torch.float32).min
    b = torch.full((m,), low, device="cuda:0")
    b[m // 2:] = -low
    for act in range(1, 5):
        out = binding.fold_epilogue(binding.FORMAT_Q4K, w, m, k, q, ds, b, act).cpu()
        assert not out.isnan().any() and (out[:, :m // 2] == 0).all() and (out[:, m // 2:] > 1e38).all(), act


@pytest.mark.parametrize("fmt,n", [(binding.FORMAT_Q4K, 3), (binding.FORMAT_Q4K, 40), (binding.FORMAT_Q4K, 150),
                                   (binding.FORMAT_Q4K_REPACKED, 11), (binding.FORMAT_Q6K, 4),
                                   (binding.FORMAT_Q6K, 150)])
@pytest.mark.parametrize("m,pad", [(96, 32), (97, 30), (96, 2)])
def test_strided_outputs_in_place_residual(fmt, n, m, pad):
    """Output rows as a slice of a wider array that is its own residual; the
    columns beside it are left as they were."""
    k = 512
    w, q, ds = _setup(fmt, 7, m, k, n)
    fold = (binding.fold_epilogue if _own(fmt, m, n) else _plain)(fmt, w, m, k, q, ds).cpu().numpy()
    rng = np.random.default_rng(9)
    r = rng.standard_normal((n, m)).astype(np.float32)
    wide = torch.full((n, m + pad), 5.0, device="cuda:0")
    out = wide[:, :m]
    out.copy_(to_dev(r))
    note("epilogue strided fmt=%d n=%d m=%d pad=%d" % (fmt, n, m, pad))
    got = binding.fold_epilogue(fmt, w, m, k, q, ds, residual=out, out=out)
    torch.cuda.synchronize()
    assert got is out and (wide[:, m:] == 5).all()
    refs.check_epilogue(out.cpu().numpy(), fold, None, 0, r, False, "in place")


def test_epilogue_row_split_launch():
    """A prefill shape that the binary16 kernel cuts into a 128-token and a
    64-token part: both parts read their rows of bias and residual."""
    _case(binding.FORMAT_Q4K, 11008, 256, 512, binding.ACT_RELU, np.float32, False)


def test_epilogue_keeps_nan_and_infinities_of_the_residual():
    """ReLU of NaN is NaN; the residual is added as it is."""
    m, k, n = 64, 256, 20
    w, q, ds = _setup(binding.FORMAT_Q4K, 31, m, k, n)
    b = np.zeros(m, np.float32)
    b[3], b[5], b[7] = np.nan, np.inf, -np.inf
    r = np.zeros((n, m), np.float32)
    r[:, 9], r[:, 11] = np.inf, np.nan
    note("epilogue nan")
    out = binding.fold_epilogue(binding.FORMAT_Q4K, w, m, k, q, ds, to_dev(b), binding.ACT_RELU, to_dev(r))
    torch.cuda.synchronize()
    out = out.cpu().numpy()
    assert np.isnan(out[:, 3]).all() and (out[:, 5] == np.inf).all() and (out[:, 7] == 0).all()
    assert (out[:, 9] == np.inf).all() and np.isnan(out[:, 11]).all()
    keep = [c for c in range(m) if c not in (3, 5, 7, 9, 11)]
    assert np.isfinite(out[:, keep]).all()


@pytest.mark.parametrize("fmt,m,n", [(binding.FORMAT_Q4K, 300, 3), (binding.FORMAT_Q4K, 300, 200),
                                     (binding.FORMAT_Q6K, 300, 30), (binding.FORMAT_Q6K, 4200, 30),
                                     (binding.FORMAT_Q6K, 300, 100)])
def test_epilogue_on_two_streams_and_in_a_graph(fmt, m, n):
    k = 1024
    w, q, ds = _setup(fmt, 32, m, k, n)
    bias = torch.randn(m, device=w.device)
    x = torch.randn(n, m, device=w.device)
    call = lambda out: binding.fold_epilogue(fmt, w, m, k, q, ds, bias, binding.ACT_GELU, x, out=out)
    note("epilogue streams fmt=%d m=%d n=%d" % (fmt, m, n))
    ref, out = call(None), torch.zeros(n, m, device=w.device)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            a = call(None)
        b = call(None)
        torch.cuda.synchronize()
        assert torch.equal(a, ref) and torch.equal(b, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for i in range(4):
        x.copy_(torch.randn(n, m, device=w.device))
        g.replay()
        eager = call(None)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


def test_epilogue_binding_refusals():
    m, k, n = 32, 256, 4
    w, q, ds = _setup(binding.FORMAT_Q4K, 1, m, k, n)
    call = lambda **kw: binding.fold_epilogue(binding.FORMAT_Q4K, w, m, k, q, ds, **kw)  # noqa: E731
    with pytest.raises(ValueError):
        call(bias=torch.zeros(m + 1, device="cuda:0"))
    with pytest.raises(TypeError):
        call(bias=torch.zeros(m, device="cuda:0", dtype=torch.float16))
    with pytest.raises(ValueError):
        call(residual=torch.zeros(n, m + 1, device="cuda:0"))
    with pytest.raises(ValueError):
        call(residual=torch.zeros(m, n, device="cuda:0").t())
    with pytest.raises(ValueError):
        call(residual=torch.zeros(1, m, device="cuda:0").expand(n, m))
    with pytest.raises(TypeError):
        call(out=torch.zeros(n, m, device="cuda:0"), f16=True)
    with pytest.raises(binding.MMQError):
        call(activation=9)
    with pytest.raises(ValueError):
        binding.fold_epilogue(binding.FORMAT_Q6K, w, m, k, q, ds)
    with pytest.raises(TypeError):
        binding.fold_epilogue(binding.FORMAT_Q4K_TILES, w, m, k, q, ds)
