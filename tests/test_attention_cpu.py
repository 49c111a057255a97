"""Argument checks of the rotary, cache and attention calls without a GPU: the
C ABI rejects bad arguments before any HIP call (fake addresses, never
dereferenced), and the binding rejects what the sizes do not fit."""
import ctypes
import os

import numpy as np
import pytest
import torch

import attention_refs as refs
from q4_q8_integer_amd import binding as b

OK, NULL, SHAPE, ALIGN, OVERFLOW, DEVICE, KERNEL = 0, -1, -2, -3, -4, -5, -7
A = 0x10000
MIS = A + 4
NO_GPU = not torch.cuda.is_available()
GOOD = DEVICE if NO_GPU else None     # a good call would launch where there is a GPU


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(b.LIB_PATH):
        from q4_q8_integer_amd.build import build_library
        build_library()
    return b.load_library()


def rope(**kw):
    a = b.RopeArgs(positions=A, freq=A, axes=1, pairs=16, scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def cache(**kw):
    a = b.CacheArgs(data=A, pages=8, heads=2, head_dim=64, page=16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def plan(**kw):
    a = b.PlanArgs(table=A, lengths=A, offsets=A, seqs=3, width=4)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def query(**kw):
    a = b.QueryArgs(q=A, out=A, n=5, most=2, heads=4, scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def refused(call, want):
    if want == DEVICE and not NO_GPU:
        pytest.skip("a good call would launch")
    assert call() == want


@pytest.mark.parametrize("args,over,want", [
    ({}, {}, DEVICE), ({}, dict(dim=1024, heads=1), DEVICE), ({}, dict(n=(1 << 24) - 1), DEVICE),
    (None, {}, NULL), ({}, dict(n=-1), SHAPE), ({}, dict(heads=-1), SHAPE), ({}, dict(dim=0), SHAPE),
    (dict(pairs=0), {}, SHAPE), (dict(pairs=33), {}, SHAPE), (dict(pairs=32), {}, DEVICE), (dict(axes=0), {}, SHAPE),
    (dict(axes=3, positions_stride=2), {}, SHAPE), ({}, dict(xs=127), SHAPE), ({}, dict(os=127), SHAPE),
    ({}, dict(xs=-1), SHAPE), ({}, dict(out=A, x=A, os=200), SHAPE),
    ({}, dict(dim=1025), OVERFLOW), ({}, dict(n=1 << 24), OVERFLOW), ({}, dict(heads=1 << 31), OVERFLOW),
    ({}, dict(xs=1 << 41), OVERFLOW), (dict(positions_stride=1 << 41), {}, OVERFLOW),
    (dict(positions=0), {}, NULL), (dict(freq=0), {}, NULL), ({}, dict(x=0), NULL), ({}, dict(out=0), NULL),
    (dict(positions=MIS), {}, ALIGN), (dict(freq=MIS), {}, ALIGN), (dict(axis=MIS), {}, ALIGN), ({}, dict(x=MIS), ALIGN),
    ({}, dict(out=MIS), ALIGN), (dict(positions=0), dict(n=0, x=0), OK), (dict(positions=0), dict(heads=0, x=0), OK),
])
def test_rope_refusals(lib, args, over, want):
    a = dict(x=A, xs=0, half=0, n=4, heads=2, dim=64, out=2 * A, os=0)
    a.update(over)
    refused(lambda: lib.rope_rows(None if args is None else rope(**args), *a.values(), None), want)


CACHE = [(dict(pages=0), SHAPE), (dict(heads=0), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=48), SHAPE),
         (dict(head_dim=288), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=2048), SHAPE),
         (dict(page=-16), SHAPE), (dict(format=2), KERNEL), (dict(format=-1), KERNEL), (dict(pages=1 << 31), OVERFLOW),
         (dict(heads=1025), OVERFLOW), (dict(pages=1 << 30, heads=1024), OVERFLOW)]
PLAN = [(dict(seqs=-1), SHAPE), (dict(width=0), SHAPE), (dict(width=-1), SHAPE), (dict(table_stride=3), SHAPE),
        (dict(offsets=0), SHAPE), (dict(seqs=65536), OVERFLOW), (dict(width=(1 << 26) + 1), OVERFLOW),
        (dict(table_stride=1 << 41), OVERFLOW)]
LATE = [(dict(data=0), {}, NULL), (dict(data=MIS), {}, ALIGN), ({}, dict(table=0), NULL), ({}, dict(lengths=0), NULL),
        ({}, dict(table=MIS), ALIGN), ({}, dict(lengths=MIS), ALIGN), ({}, dict(offsets=MIS), ALIGN)]
BOTH = [(c, {}, w) for c, w in CACHE] + [({}, p, w) for p, w in PLAN] + LATE + [
    ({}, {}, DEVICE), ({}, dict(seqs=65535, width=1 << 26), DEVICE), (dict(pages=(1 << 31) - 1, heads=1, head_dim=32, format=1), {}, OVERFLOW),
    (dict(head_dim=256, page=1024, format=1), {}, DEVICE), ({}, dict(seqs=0, table=0), OK)]


@pytest.mark.parametrize("c,p,want", BOTH)
def test_cache_and_plan_refusals(lib, c, p, want):
    refused(lambda: lib.kv_write(cache(**c), plan(**p), None, A, A, 0, 5, 0, 0, None), want)
    refused(lambda: lib.kv_read(cache(**c), plan(**p), A, A, 0, 5, 0, 0, None), want)
    if want not in (OVERFLOW, DEVICE):
        assert lib.kv_attend(cache(**c), plan(**p), query(), A, 1 << 40, None) == want


@pytest.mark.parametrize("over,want", [
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(k=MIS), ALIGN), (dict(v=MIS), ALIGN), (dict(n=-1), SHAPE),
    (dict(n=1 << 24), OVERFLOW), (dict(ks=127), SHAPE), (dict(vs=127), SHAPE), (dict(ks=-5), SHAPE), (dict(vs=1 << 41), OVERFLOW),
    (dict(n=0, k=0, v=0), OK),
])
def test_rows_refusals(lib, over, want):
    a = dict(k=A, v=A, half=0, n=5, ks=0, vs=0)
    a.update(over)
    assert lib.kv_write(cache(), plan(), None, *a.values(), None) == want
    assert lib.kv_read(cache(), plan(), *a.values(), None) == want


def test_write_refuses_a_bad_rotation(lib):
    for r, want in ((dict(pairs=33), SHAPE), (dict(pairs=0), SHAPE), (dict(axes=0), SHAPE), (dict(freq=0), NULL),
                    (dict(positions=MIS), ALIGN)):
        assert lib.kv_write(cache(), plan(), rope(**r), A, A, 0, 5, 0, 0, None) == want
    assert lib.kv_write(None, plan(), None, A, A, 0, 5, 0, 0, None) == NULL
    assert lib.kv_write(cache(), None, None, A, A, 0, 5, 0, 0, None) == NULL


@pytest.mark.parametrize("c,p,over,want", [
    ({}, {}, dict(heads=3), SHAPE), ({}, {}, dict(heads=0), SHAPE), ({}, {}, dict(window=-1), SHAPE), ({}, {}, dict(most=0), SHAPE),
    ({}, {}, dict(q_stride=255), SHAPE), ({}, {}, dict(out_stride=255), SHAPE), ({}, {}, dict(n=-1), SHAPE),
    ({}, {}, dict(n=1 << 24), OVERFLOW), ({}, {}, dict(heads=64 * 2, n=1 << 22, most=1 << 22), OVERFLOW),
    ({}, dict(width=1 << 26), dict(n=100000, most=100000, heads=16), OVERFLOW),
    ({}, {}, dict(q=0), NULL), ({}, {}, dict(out=0), NULL), ({}, {}, dict(q=MIS), ALIGN), ({}, {}, dict(out=MIS), ALIGN),
    ({}, {}, dict(lse=MIS), ALIGN), ({}, {}, dict(n=0, most=0, q=0), OK), ({}, {}, {}, DEVICE),
    ({}, dict(width=1 << 26, seqs=65535), {}, DEVICE),
])
def test_attend_refusals(lib, c, p, over, want):
    refused(lambda: lib.kv_attend(cache(**c), plan(**p), query(**over), A, 1 << 40, None), want)


def test_attend_workspace(lib):
    n = ctypes.c_int64(-1)
    assert lib.kv_attend_workspace(cache(), plan(), query(), n) == OK and n.value == 0      # 64 tokens at most: not split
    assert lib.kv_attend_workspace(cache(), plan(width=100), query(), n) == OK and n.value > 0
    for space, size, want in ((0, n.value, NULL), (MIS, n.value, ALIGN), (A, n.value - 1, SHAPE)):
        assert lib.kv_attend(cache(), plan(width=100), query(), space, size, None) == want
    assert lib.kv_attend_workspace(cache(), plan(), query(), None) == NULL
    assert lib.kv_attend_workspace(cache(), plan(), None, n) == NULL
    assert lib.kv_attend_workspace(cache(), plan(), query(heads=3), n) == SHAPE
    assert lib.kv_attend_workspace(cache(), plan(), query(n=0), n) == OK and n.value == 0


@pytest.mark.parametrize("dim,page,bits", [(64, 16, 8), (128, 64, 4), (96, 32, 8), (256, 1024, 4), (32, 16, 4)])
def test_cache_bytes(lib, dim, page, bits):
    want = refs.record_parts(dim, page, bits)[-1]
    assert b.cache_bytes(5, 3, dim, page, b.KV_Q8 if bits == 8 else b.KV_Q4) == 15 * want
    n = ctypes.c_int64()
    assert lib.kv_cache_bytes(cache(data=0), n) == OK
    assert lib.kv_cache_bytes(cache(), None) == NULL and lib.kv_cache_bytes(None, n) == NULL


def test_struct_layouts():
    # as a C compiler lays out the structs of include/mmq.h on x86-64
    assert ctypes.sizeof(b.RopeArgs) == 48 and b.RopeArgs.scale.offset == 44
    assert ctypes.sizeof(b.CacheArgs) == 32 and b.CacheArgs.format.offset == 28
    assert ctypes.sizeof(b.PlanArgs) == 48 and b.PlanArgs.table_stride.offset == 40
    assert ctypes.sizeof(b.QueryArgs) == 80 and b.QueryArgs.scale.offset == 72


def test_binding_refuses_cpu_tensors():
    x, i = torch.zeros(3, 128), torch.zeros(3, dtype=torch.int32)
    c = b.KVCache(torch.zeros(2, 2, 2 * 16 * 68, dtype=torch.uint8), 64, 16)
    p = b.KVPlan(torch.zeros(3, 1, dtype=torch.int32), i)
    for call in (lambda: b.rope(x, 2, b.Rope(i, torch.ones(8))), lambda: b.kv_write(c, p, x, x), lambda: b.kv_read(c, p, 3),
                 lambda: b.kv_attend(c, p, x, 2), lambda: b.kv_attend(None, p, x, 2), lambda: b.new_cache(2, 2, 60, 16)):
        with pytest.raises((TypeError, ValueError, b.MMQError)):
            call()


@pytest.mark.parametrize("dim", [32, 96, 128, 256])
@pytest.mark.parametrize("bits", [8, 4])
def test_layout_reference_round_trip(dim, bits):
    """The tests' own packing: every code has a place of its own, and comes back."""
    rng = np.random.default_rng(dim)
    for place, key in ((refs.key_place(dim), True), (refs.value_place(dim), False)):
        assert sorted(place) == list(range(dim))
        code = rng.integers(-7, 8, dim)
        got = refs.code_bytes(code, place, bits, key)
        assert got.shape == (dim * bits // 8,) and np.array_equal(refs.byte_codes(got, place, bits, key), code)


@pytest.mark.parametrize("seqs,n,most,width,cut", [
    (1, 2048, 2048, 100, False), (1, 2048, 2048, 1 << 14, False),   # one sequence's tiles fill the chip
    (64, 575, 512, 100, True), (4, 515, 512, 2048, True), (8, 4096, 512, 2048, True), (64, 64, 64, 64, True),   # of several
    (1, 512, 512, 100, True), (64, 64, 1, 16, False), (1, 1, 1, 16, True)])
def test_what_is_cut(lib, seqs, n, most, width, cut):
    """8 heads of 128 with 4 query heads each: several sequences on a table past
    1280 tokens are cut, however many tiles they may have, as their lengths may differ."""
    c = cache(pages=1 << 20, heads=8, head_dim=128, page=64, data=0)
    size = ctypes.c_int64(-1)
    q = query(n=n, most=most, heads=32, q_half=1, out_half=1)
    assert lib.kv_attend_workspace(c, plan(seqs=seqs, width=width), q, size) == OK
    assert (size.value > 0) == cut
