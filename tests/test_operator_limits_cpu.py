"""Sizes at the borders of the operators' limits, through the C ABI without a
GPU: what the header allows reaches the device check, what it excludes does
not (fake addresses, never dereferenced)."""
import os

import pytest
import torch

from q4_q8_integer_amd import binding

OK, OVERFLOW, DEVICE = 0, -4, -5
A = 0x10000

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="without a GPU only: good calls would launch")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from q4_q8_integer_amd.build import build_library
        build_library()
    return binding.load_library()


def grouped(lib, fmt, experts, m, k, tokens, slots, f16=1):
    e = binding.Epilogue(out_f16=f16)
    return lib.mmq_fold_grouped(fmt, A, experts, m, k, A, A, tokens, A, A, slots, e, A, None)


@pytest.mark.parametrize("fmt", [binding.FORMAT_Q4K, binding.FORMAT_Q6K])
def test_grouped_limits(lib, fmt):
    assert grouped(lib, fmt, 2, 16384, 256, 64, 1 << 21) == DEVICE             # slots*m = 2^35
    assert grouped(lib, fmt, 8, 1 << 20, 256, 64, (1 << 20) - 1) == DEVICE     # just below 2^40
    assert grouped(lib, fmt, 8, 1 << 20, 256, 64, 1 << 20) == OVERFLOW         # slots*m = 2^40
    assert grouped(lib, fmt, 1, 512, 256, 64, (1 << 31) - 1) == DEVICE
    assert grouped(lib, fmt, 4096, 8 << 17, 256, 64, 64) == DEVICE             # 2^32 rows of weights
    assert grouped(lib, fmt, 4096, 8 << 18, 256, 64, 64) == OVERFLOW           # 2^33: past 2^40 bytes
    assert grouped(lib, fmt, 2, 64, 256, (1 << 24) - 1, 64) == DEVICE          # tokens*k just below 2^32
    assert grouped(lib, fmt, 2, 64, 256, 1 << 24, 64) == OVERFLOW


def combine(lib, f16, slots, m, n, top=2):
    return lib.moe_combine(A, f16, slots, m, A, A, n, top, 0, A, None)


def test_combine_limits(lib):
    assert combine(lib, 1, 64, 4096, 1 << 20) == DEVICE          # 2 workgroups a token
    assert combine(lib, 1, 64, 4096, (1 << 23) - 1) == DEVICE
    assert combine(lib, 1, 64, 4096, 1 << 23) == OVERFLOW        # 2^24 workgroups
    assert combine(lib, 0, 64, 4096, (1 << 22) - 1) == DEVICE
    assert combine(lib, 0, 64, 4096, 1 << 22) == OVERFLOW
    assert combine(lib, 1, 64, 100, (1 << 24) - 1) == DEVICE     # 4 values over: a value per thread
    assert combine(lib, 1, 64, 4097, 1 << 20) == OVERFLOW        # 17 workgroups a token
    assert combine(lib, 0, 64, 64, (1 << 24) - 1, top=64) == DEVICE
    assert combine(lib, 0, 64, 64, 1 << 24, top=64) == OVERFLOW
    for m in ((1 << 31) - 1, (1 << 31) - 4, (1 << 31) - 8):      # columns up to the last int
        assert combine(lib, 0, 1, m, 1, 1) == DEVICE
        assert combine(lib, 1, 1, m, 1, 1) == DEVICE


def test_route_limits(lib):
    def route(n, experts, top):
        return lib.moe_route(A, n, experts, 0, top, 1, 1.0, A, A, A, A, A, None)
    assert route((1 << 26) - 4, 2, 1) == DEVICE
    for more in (3, 2, 1, 0):                       # 2^24 workgroups of 4 waves
        assert route((1 << 26) - more, 2, 1) == OVERFLOW
    assert route(1 << 24, 64, 64) == DEVICE         # 2^30 choices
    assert route((1 << 24) + 1, 64, 64) == OVERFLOW
    assert route(5, 1024, 64) == DEVICE
