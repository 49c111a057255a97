"""Argument checks of the epilogue, grouped, router, combine and norm calls:
the C ABI rejects bad arguments before any HIP call (fake addresses, never
dereferenced), and the binding rejects tensors that do not hold what the
sizes say."""
import ctypes
import os

import pytest
import torch

from q4_q8_integer_amd import binding

OK, NULL, SHAPE, ALIGN, OVERFLOW, DEVICE, KERNEL = 0, -1, -2, -3, -4, -5, -7
A = 0x10000
MIS = A + 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from q4_q8_integer_amd.build import build_library
        build_library()
    return binding.load_library()


def epi(**kw):
    e = binding.Epilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def norm(**kw):
    a = binding.Norm(x=A, weight=A, residual_scale=1.0, eps=1e-5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(fmt=6), KERNEL), (dict(fmt=-1), KERNEL),
    (dict(e=dict(activation=5)), KERNEL), (dict(e=dict(activation=-1)), KERNEL),
    (dict(e=dict(out_stride=31)), SHAPE), (dict(e=dict(residual=A, residual_stride=31)), SHAPE),
    (dict(e=dict(out_stride=-1)), SHAPE), (dict(e=dict(out_stride=1 << 41)), OVERFLOW),
    (dict(e=dict(bias=MIS)), ALIGN), (dict(e=dict(residual=MIS)), ALIGN),
    (dict(e=None), NULL), (dict(w=0), NULL), (dict(q=0), NULL), (dict(ds=0), NULL), (dict(out=0), NULL),
    (dict(w=MIS), ALIGN), (dict(q=MIS), ALIGN), (dict(ds=MIS), ALIGN), (dict(out=MIS), ALIGN),
    (dict(k=128), SHAPE), (dict(k=0), SHAPE), (dict(m=-1), SHAPE), (dict(n=-1), SHAPE),
    (dict(k=(1 << 24) + 256), OVERFLOW), (dict(m=1 << 31), OVERFLOW), (dict(n=1 << 31), OVERFLOW),
    (dict(n=0, w=0, q=0, ds=0, out=0), OK), (dict(m=0, w=0), OK),
])
@pytest.mark.parametrize("fmt", range(6))
def test_epilogue_refusals(lib, fmt, over, want):
    a = dict(fmt=fmt, w=A, m=32, k=256, q=A, ds=A, n=4, e={}, out=A)
    a.update(over)
    e = None if a["e"] is None else epi(**a["e"])
    assert lib.mmq_fold_epilogue(a["fmt"], a["w"], a["m"], a["k"], a["q"], a["ds"], a["n"], e, a["out"], None) == want


@pytest.mark.parametrize("over,want", [
    (dict(fmt=1), KERNEL), (dict(fmt=3), KERNEL), (dict(fmt=9), KERNEL),
    (dict(experts=0), SHAPE), (dict(experts=4097), OVERFLOW), (dict(tokens=0), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(rows=0, tokens=9), SHAPE), (dict(slots=-1), SHAPE), (dict(k=100), SHAPE), (dict(m=-8), SHAPE),
    (dict(tokens=1 << 24, k=256), OVERFLOW), (dict(m=1 << 31), OVERFLOW), (dict(slots=1 << 31), OVERFLOW),
    (dict(experts=4096, m=1 << 23, k=1 << 13), OVERFLOW),
    (dict(w=0), NULL), (dict(q=0), NULL), (dict(ds=0), NULL), (dict(offsets=0), NULL), (dict(out=0), NULL),
    (dict(e=None), NULL), (dict(e=dict(activation=7)), KERNEL), (dict(e=dict(out_stride=8)), SHAPE),
    (dict(w=MIS), ALIGN), (dict(q=MIS), ALIGN), (dict(ds=MIS), ALIGN), (dict(offsets=MIS), ALIGN),
    (dict(rows=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(e=dict(bias=MIS)), ALIGN),
    (dict(fmt=2, m=4), ALIGN),          # 4 * 210 bytes: the second expert's rows would start off a 16-byte boundary
    (dict(slots=0, w=0, q=0, ds=0, offsets=0, out=0), OK), (dict(m=0, w=0, offsets=0), OK),
])
def test_grouped_refusals(lib, over, want):
    a = dict(fmt=0, w=A, experts=3, m=32, k=256, q=A, ds=A, tokens=4, rows=A, offsets=A, slots=10, e={}, out=A)
    a.update(over)
    e = None if a["e"] is None else epi(**a["e"])
    assert lib.mmq_fold_grouped(a["fmt"], a["w"], a["experts"], a["m"], a["k"], a["q"], a["ds"], a["tokens"],
                                a["rows"], a["offsets"], a["slots"], e, a["out"], None) == want


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), SHAPE), (dict(experts=0), SHAPE), (dict(top=0), SHAPE), (dict(top=9), SHAPE), (dict(stride=7), SHAPE),
    (dict(experts=1025), OVERFLOW), (dict(experts=100, top=65), OVERFLOW), (dict(n=1 << 30), OVERFLOW),
    (dict(n=1 << 31), OVERFLOW),
    (dict(logits=0), NULL), (dict(ids=0), NULL), (dict(weights=0), NULL), (dict(slot=0), NULL), (dict(rows=0), NULL),
    (dict(offsets=0), NULL), (dict(logits=MIS), ALIGN), (dict(ids=MIS), ALIGN), (dict(weights=MIS), ALIGN),
    (dict(slot=MIS), ALIGN), (dict(rows=MIS), ALIGN), (dict(offsets=MIS), ALIGN),
    (dict(n=0, logits=0, ids=0), OK),
])
def test_route_refusals(lib, over, want):
    a = dict(logits=A, n=5, experts=8, stride=0, top=2, normalize=1, scale=1.0, ids=A, weights=A, slot=A, rows=A,
             offsets=A)
    a.update(over)
    assert lib.moe_route(*a.values(), None) == want


@pytest.mark.parametrize("over,want", [
    (dict(slots=-1), SHAPE), (dict(m=-1), SHAPE), (dict(n=-1), SHAPE), (dict(top=0), SHAPE),
    (dict(top=65), OVERFLOW), (dict(slots=1 << 31), OVERFLOW), (dict(n=1 << 31), OVERFLOW), (dict(m=1 << 31), OVERFLOW),
    (dict(n=1 << 29, top=4), OVERFLOW), (dict(n=1 << 24, m=1 << 16), OVERFLOW),
    (dict(y=0), NULL), (dict(slot=0), NULL), (dict(weights=0), NULL), (dict(out=0), NULL),
    (dict(y=MIS), ALIGN), (dict(slot=MIS), ALIGN), (dict(weights=MIS), ALIGN), (dict(residual=MIS), ALIGN),
    (dict(out=MIS), ALIGN), (dict(n=0, y=0, out=0), OK), (dict(m=0, y=0, out=0), OK),
])
def test_combine_refusals(lib, over, want):
    a = dict(y=A, f16=0, slots=8, m=16, slot=A, weights=A, n=4, top=2, residual=0, out=A)
    a.update(over)
    assert lib.moe_combine(*a.values(), None) == want


@pytest.mark.parametrize("over,args,want", [
    (dict(n=-1), {}, SHAPE), (dict(k=0), {}, SHAPE), (dict(k=48), {}, SHAPE), (dict(k=(1 << 24) + 32), {}, OVERFLOW),
    (dict(n=1 << 31), {}, OVERFLOW), (dict(n=1 << 23), {}, OVERFLOW),
    (dict(q=0), {}, NULL), (dict(ds=0), {}, NULL), ({}, dict(x=0), NULL), ({}, dict(weight=0), NULL),
    ({}, dict(y=A), NULL), ({}, dict(r=A), NULL), ({}, dict(gate=A), NULL), ({}, dict(y_weight=A), NULL),
    ({}, dict(residual_scale=0.5), NULL),
    ({}, dict(x_stride=32), SHAPE), ({}, dict(y=A, r=A, y_stride=63), SHAPE), ({}, dict(y=A, r=A, r_stride=8), SHAPE),
    ({}, dict(y=A, r=A, gate=A, gate_stride=32), SHAPE), ({}, dict(x_stride=1 << 41), OVERFLOW),
    ({}, dict(x=MIS), ALIGN), ({}, dict(weight=MIS), ALIGN), ({}, dict(h=MIS), ALIGN), ({}, dict(y=MIS, r=A), ALIGN),
    ({}, dict(y=A, r=MIS), ALIGN), ({}, dict(y=A, r=A, gate=MIS), ALIGN), ({}, dict(y=A, r=A, y_weight=MIS), ALIGN),
    (dict(q=MIS), {}, ALIGN), (dict(ds=MIS), {}, ALIGN),
    ({}, dict(x_stride=66), ALIGN), ({}, dict(y=A, r=A, y_f16=1, y_stride=68), ALIGN),
    ({}, dict(y=A, r=A, r_stride=65), ALIGN),
    (dict(n=0, q=0), dict(x=0), OK),
])
def test_norm_refusals(lib, over, args, want):
    a = dict(n=4, k=64, q=A, ds=A)
    a.update(over)
    assert lib.q8_quantize_norm(norm(**args), a["n"], a["k"], a["q"], a["ds"], None) == want
    if a["k"] == 64:   # operand tiles take k in whole super-blocks only
        assert lib.q8_quantize_norm_tiled(norm(**args), a["n"], 64, a["q"], a["ds"], None) == SHAPE


def test_norm_refusals_more(lib):
    assert lib.q8_quantize_norm(None, 4, 64, A, A, None) == NULL
    assert lib.residual_norm(norm(), 4, 64, None) == NULL            # h is what it is called for
    assert lib.residual_norm(norm(h=MIS), 4, 64, None) == ALIGN
    assert lib.q8_quantize_norm_tiled(norm(), 4, 256, 0, A, None) == NULL
    assert lib.residual_norm(norm(), 0, 64, None) == OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a GPU only")
def test_good_calls_reach_the_device_check(lib):
    e = epi()
    for fmt in range(6):
        assert lib.mmq_fold_epilogue(fmt, A, 32, 256, A, A, 4, e, A, None) == DEVICE
    assert lib.mmq_fold_grouped(0, A, 3, 32, 256, A, A, 4, A, A, 10, e, A, None) == DEVICE
    assert lib.mmq_fold_grouped(2, A, 3, 32, 256, A, A, 10, 0, A, 10, e, A, None) == DEVICE
    assert lib.moe_route(A, 5, 8, 0, 2, 1, 1.0, A, A, A, A, A, None) == DEVICE
    assert lib.moe_combine(A, 0, 8, 16, A, A, 4, 2, 0, A, None) == DEVICE
    assert lib.q8_quantize_norm(norm(), 4, 64, A, A, None) == DEVICE
    assert lib.residual_norm(norm(h=A, y=A, r=A), 4, 64, None) == DEVICE


def test_struct_layouts():
    # as a C compiler lays out the structs of include/mmq.h on x86-64
    assert ctypes.sizeof(binding.Epilogue) == 48 and binding.Epilogue.activation.offset == 32
    assert ctypes.sizeof(binding.Norm) == 104 and binding.Norm.residual_scale.offset == 88


def test_binding_refuses_cpu_tensors_and_shapes():
    x = torch.zeros(4, 64)
    with pytest.raises((TypeError, ValueError)):
        binding.quantize_norm(x, torch.ones(64))
    with pytest.raises((TypeError, ValueError)):
        binding.route(torch.zeros(4, 8), 2)
    with pytest.raises((TypeError, ValueError)):
        binding.combine(torch.zeros(8, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises((TypeError, ValueError)):
        binding.fold_epilogue(9, x, 4, 256, x, x)
    with pytest.raises((TypeError, ValueError)):
        binding.fold_grouped(1, x, 2, 4, 256, x, x, x)
