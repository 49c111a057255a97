"""Thin ctypes binding over the C ABI of ``include/mmq.h``.

Argument marshalling only: torch tensors give device pointers and the current
HIP stream; every step of the computation runs in the HIP kernels of
``libq4q8mmq.so``.  There is no fallback: if the library is missing or the
device is not gfx950, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4q8mmq.so")
EXPORTS = ("q8_quantize_rows", "q8_quantize_silu_mul", "mmq_q4k_q8", "mmq_q4k_q8_fp32out", "mmq_q4k_q8_f16out",
           "mmq_q4k_q8_fold", "mmq_q6k_q8", "mmq_q6k_q8_fp32out", "mmq_q6k_q8_f16out", "mmq_q6k_q8_fold",
           "q4k_repack", "mmq_q4kr_q8_fp32out", "q8_quantize_rows_tiled", "mmq_q4k_q8t_fp32out",
           "mmq_q4kr_q8t_fp32out", "mmq_q6k_q8t_fp32out", "q8_quantize_silu_mul_tiled",
           "mmq_kernel_choice", "mmq_status_string", "mmq_fold_epilogue", "mmq_fold_grouped", "moe_route",
           "moe_combine", "q8_quantize_norm", "q8_quantize_norm_tiled", "residual_norm", "rope_rows", "kv_cache_bytes",
           "kv_write", "kv_read", "kv_attend_workspace", "kv_attend")

# enum mmq_kernel / enum mmq_format of include/mmq.h
KERNEL_AUTO, KERNEL_DOT4, KERNEL_FEW, KERNEL_F16, KERNEL_I8, KERNEL_NARROW, KERNEL_STREAM = 0, 1, 2, 3, 4, 5, 6
KERNEL_NAMES = {KERNEL_DOT4: "dot4", KERNEL_FEW: "few", KERNEL_F16: "f16", KERNEL_I8: "i8",
                KERNEL_NARROW: "narrow", KERNEL_STREAM: "stream"}
(FORMAT_Q4K, FORMAT_Q4K_REPACKED, FORMAT_Q6K, FORMAT_Q4K_TILES, FORMAT_Q4K_REPACKED_TILES,
 FORMAT_Q6K_TILES) = range(6)
_FORMAT_NAMES = {FORMAT_Q4K: "q4k", FORMAT_Q4K_REPACKED: "repacked", FORMAT_Q6K: "q6k", FORMAT_Q4K_TILES: "q4k",
                 FORMAT_Q4K_REPACKED_TILES: "repacked", FORMAT_Q6K_TILES: "q6k"}
_TILE_FORMATS = (FORMAT_Q4K_TILES, FORMAT_Q4K_REPACKED_TILES, FORMAT_Q6K_TILES)
# enum mmq_activation
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = range(5)
# enum kv_format
KV_Q8, KV_Q4 = range(2)
Q4K_BLOCK_BYTES, Q6K_BLOCK_BYTES, REPACK_RECORD_BYTES = 144, 210, 2368
_MMQ_CALLS = ("mmq_q4k_q8", "mmq_q4k_q8_fp32out", "mmq_q4k_q8_f16out",
              "mmq_q6k_q8", "mmq_q6k_q8_fp32out", "mmq_q6k_q8_f16out", "mmq_q4kr_q8_fp32out",
              "mmq_q4k_q8t_fp32out", "mmq_q4kr_q8t_fp32out", "mmq_q6k_q8t_fp32out")
_lib = None


class Epilogue(ctypes.Structure):
    """mmq_epilogue of include/mmq.h."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("activation", ctypes.c_int), ("residual_f16", ctypes.c_int),
                ("out_f16", ctypes.c_int)]


class Norm(ctypes.Structure):
    """q8_norm of include/mmq.h."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("y_weight", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("r", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64), ("r_stride", ctypes.c_int64), ("residual_scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("y_f16", ctypes.c_int)]


class RopeArgs(ctypes.Structure):
    """rope_plan of include/mmq.h."""
    _fields_ = [("positions", ctypes.c_void_p), ("freq", ctypes.c_void_p), ("axis", ctypes.c_void_p),
                ("positions_stride", ctypes.c_int64), ("axes", ctypes.c_int), ("pairs", ctypes.c_int),
                ("adjacent", ctypes.c_int), ("scale", ctypes.c_float)]


class CacheArgs(ctypes.Structure):
    """kv_cache of include/mmq.h."""
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page", ctypes.c_int), ("format", ctypes.c_int)]


class PlanArgs(ctypes.Structure):
    """kv_plan of include/mmq.h."""
    _fields_ = [("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("seqs", ctypes.c_int64), ("width", ctypes.c_int64), ("table_stride", ctypes.c_int64)]


class QueryArgs(ctypes.Structure):
    """kv_query of include/mmq.h."""
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("n", ctypes.c_int64),
                ("most", ctypes.c_int64), ("heads", ctypes.c_int), ("q_half", ctypes.c_int), ("out_half", ctypes.c_int),
                ("window", ctypes.c_int), ("scale", ctypes.c_float)]


class Rope(NamedTuple):
    """Rotary positions of the rows of a call (rope_plan): pair j of a head
    turns by positions[row, axis[j]] * freq[j]."""
    positions: torch.Tensor            # int32 [n] or [n, axes]
    freq: torch.Tensor                 # float32 [pairs], radians per position
    axis: Optional[torch.Tensor] = None   # int32 [pairs], or None: axis 0
    adjacent: bool = False             # pairs (2 j, 2 j + 1), else (j, pairs + j)
    scale: float = 1.0                 # of cosine and sine


class KVCache(NamedTuple):
    """A paged cache of quantised keys and values; new_cache makes one."""
    data: torch.Tensor                 # uint8 [pages, heads, bytes of a record]
    head_dim: int
    page: int                          # tokens of a page
    format: int = KV_Q8


class KVPlan(NamedTuple):
    """Which row of a call is which token of which sequence (kv_plan): rows
    offsets[s] .. offsets[s + 1] - 1 are the last of sequence s, lengths[s]
    long with them; without offsets row s is the last token of sequence s."""
    table: torch.Tensor                # int32 [seqs, width], page ids
    lengths: torch.Tensor              # int32 [seqs]
    offsets: Optional[torch.Tensor] = None   # int32 [seqs + 1]


class Routing(NamedTuple):
    """What route() returns."""
    ids: torch.Tensor       # int32 [n, top]
    weights: torch.Tensor   # float32 [n, top]
    slot: torch.Tensor      # int32 [n, top]
    rows: torch.Tensor      # int32 [n * top]
    offsets: torch.Tensor   # int32 [experts + 1]


class MMQError(RuntimeError):
    """A non-zero status from the C ABI."""

    def __init__(self, fn: str, status: int, text: str):
        super().__init__("%s failed: %s (status %d)" % (fn, text, status))
        self.status = status


def load_library(path: str = LIB_PATH):
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("HIP library %s is missing: build it with "
                           "`python -m q4_q8_integer_amd.build` (or __graft_entry__.build())" % path)
    lib = ctypes.CDLL(path)
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    lib.q8_quantize_rows.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.q8_quantize_rows.restype = ctypes.c_int
    lib.q8_quantize_rows_tiled.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.q8_quantize_rows_tiled.restype = ctypes.c_int
    lib.q8_quantize_silu_mul_tiled.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    lib.q8_quantize_silu_mul_tiled.restype = ctypes.c_int
    lib.q8_quantize_silu_mul.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    lib.q8_quantize_silu_mul.restype = ctypes.c_int
    lib.q4k_repack.argtypes = [vp, i64, i64, vp, vp]
    lib.q4k_repack.restype = ctypes.c_int
    for name in _MMQ_CALLS:
        fn = getattr(lib, name)
        fn.argtypes = [vp, i64, i64, vp, vp, i64, vp, vp]
        fn.restype = ctypes.c_int
    for name in ("mmq_q4k_q8_fold", "mmq_q6k_q8_fold"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, i64, i64, vp, vp, i64, vp, ctypes.c_int, ctypes.c_int, vp]
        fn.restype = ctypes.c_int
    lib.mmq_kernel_choice.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.mmq_kernel_choice.restype = ctypes.c_int
    ci, cf = ctypes.c_int, ctypes.c_float
    for name, args in (
            ("mmq_fold_epilogue", [ci, vp, i64, i64, vp, vp, i64, ctypes.POINTER(Epilogue), vp, vp]),
            ("mmq_fold_grouped", [ci, vp, i64, i64, i64, vp, vp, i64, vp, vp, i64, ctypes.POINTER(Epilogue), vp, vp]),
            ("moe_route", [vp, i64, i64, i64, ci, ci, cf, vp, vp, vp, vp, vp, vp]),
            ("moe_combine", [vp, ci, i64, i64, vp, vp, i64, ci, vp, vp, vp]),
            ("q8_quantize_norm", [ctypes.POINTER(Norm), i64, i64, vp, vp, vp]),
            ("q8_quantize_norm_tiled", [ctypes.POINTER(Norm), i64, i64, vp, vp, vp]),
            ("residual_norm", [ctypes.POINTER(Norm), i64, i64, vp]),
            ("rope_rows", [ctypes.POINTER(RopeArgs), vp, i64, ci, i64, i64, i64, vp, i64, vp]),
            ("kv_cache_bytes", [ctypes.POINTER(CacheArgs), ctypes.POINTER(i64)]),
            ("kv_write", [ctypes.POINTER(CacheArgs), ctypes.POINTER(PlanArgs), ctypes.POINTER(RopeArgs), vp, vp, ci,
                          i64, i64, i64, vp]),
            ("kv_read", [ctypes.POINTER(CacheArgs), ctypes.POINTER(PlanArgs), vp, vp, ci, i64, i64, i64, vp]),
            ("kv_attend_workspace", [ctypes.POINTER(CacheArgs), ctypes.POINTER(PlanArgs), ctypes.POINTER(QueryArgs),
                                     ctypes.POINTER(i64)]),
            ("kv_attend", [ctypes.POINTER(CacheArgs), ctypes.POINTER(PlanArgs), ctypes.POINTER(QueryArgs), vp, i64,
                           vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    lib.mmq_status_string.argtypes = [ctypes.c_int]
    lib.mmq_status_string.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().mmq_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise MMQError(fn, status, status_string(status))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %s tensor on a HIP device" % (name, dtype))


# Size checks.  The C ABI sees pointers only, so a wrong m, k or n would make
# the kernels read or write past a tensor; every wrapper below checks that
# each tensor holds what the sizes say (and that all sit on one device)
# before it calls the library, and raises ValueError otherwise.
def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _fits(t, nbytes: int, name: str):
    """A tensor argument (None passes through as NULL) holds >= nbytes bytes."""
    if t is not None and isinstance(t, torch.Tensor) and _nbytes(t) < nbytes:
        raise ValueError("%s holds %d bytes, the sizes given need %d" % (name, _nbytes(t), nbytes))


def _same_device(*ts):
    devs = {t.device for t in ts if isinstance(t, torch.Tensor)}
    if len(devs) > 1:
        raise ValueError("all tensors must be on one device, got %s" % sorted(str(d) for d in devs))


def _mmq_sizes(m: int, k: int, n: int):
    if m < 0 or n < 0 or k <= 0 or k % 256:
        raise ValueError("need m, n >= 0 and k a positive multiple of 256 (m=%d k=%d n=%d)" % (m, k, n))


def _check_fold_args(w, wbytes, m, k, q, qbytes, ds, n, out, outbytes):
    _mmq_sizes(m, k, n)
    _fits(w, wbytes, "w")
    _fits(q, qbytes, "q")
    _fits(ds, n * (k // 32) * 4, "ds")
    _fits(out, outbytes, "out")
    _same_device(w, q, ds, out)


def _w_bytes(m: int, k: int, fmt: str) -> int:
    if fmt == "q6k":
        return m * (k // 256) * Q6K_BLOCK_BYTES
    if fmt == "repacked":
        return (m + 15) // 16 * (k // 256) * REPACK_RECORD_BYTES
    return m * (k // 256) * Q4K_BLOCK_BYTES


# -------------------------------------------------------------- raw entries
# Same names and arguments as the C ABI (tensors for pointers); each checks
# that its tensors hold what the sizes say before the call.
def q8_quantize_rows(x, n, k, q, ds):
    """Enqueue the quantizer on preallocated outputs (C ABI call, same name)."""
    if n >= 0 and k > 0 and k % 32 == 0:
        _fits(x, n * k * 4, "x")
        _fits(q, n * k, "q")
        _fits(ds, n * (k // 32) * 4, "ds")
        _same_device(x, q, ds)
    _check("q8_quantize_rows", load_library().q8_quantize_rows(
        _ptr(x), n, k, _ptr(q), _ptr(ds), _stream()))


def q8_quantize_rows_tiled(x, n, k, qt, ds):
    """Enqueue the quantizer with the codes as binary16 operand tiles."""
    if n >= 0 and k > 0 and k % 256 == 0:
        _fits(x, n * k * 4, "x")
        _fits(qt, tiles_elems(n, k) * 2, "qt")
        _fits(ds, n * (k // 32) * 4, "ds")
        _same_device(x, qt, ds)
    _check("q8_quantize_rows_tiled", load_library().q8_quantize_rows_tiled(
        _ptr(x), n, k, _ptr(qt), _ptr(ds), _stream()))


def q8_quantize_silu_mul_tiled(gate, up, n, k, qt, ds):
    """Enqueue the fused SiLU-gate quantizer with the codes as operand tiles."""
    if n >= 0 and k > 0 and k % 256 == 0:
        _fits(gate, n * k * 4, "gate")
        _fits(up, n * k * 4, "up")
        _fits(qt, tiles_elems(n, k) * 2, "qt")
        _fits(ds, n * (k // 32) * 4, "ds")
        _same_device(gate, up, qt, ds)
    _check("q8_quantize_silu_mul_tiled", load_library().q8_quantize_silu_mul_tiled(
        _ptr(gate), _ptr(up), n, k, _ptr(qt), _ptr(ds), _stream()))


def q8_quantize_silu_mul(gate, up, n, k, q, ds):
    """Enqueue the fused SiLU-gate quantizer on preallocated outputs."""
    if n >= 0 and k > 0 and k % 32 == 0:
        _fits(gate, n * k * 4, "gate")
        _fits(up, n * k * 4, "up")
        _fits(q, n * k, "q")
        _fits(ds, n * (k // 32) * 4, "ds")
        _same_device(gate, up, q, ds)
    _check("q8_quantize_silu_mul", load_library().q8_quantize_silu_mul(
        _ptr(gate), _ptr(up), n, k, _ptr(q), _ptr(ds), _stream()))


def _sized(m, k, n):
    return m >= 0 and n >= 0 and k > 0 and k % 256 == 0


def mmq_q4k_q8(w, m, k, q, ds, n, dots):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q4k"), m, k, q, n * k, None, n, dots, n * m * (k // 32) * 4)
        _fits(ds, n * (k // 32) * 4, "ds")
    _check("mmq_q4k_q8", load_library().mmq_q4k_q8(
        _ptr(w), m, k, _ptr(q), _ptr(ds), n, _ptr(dots), _stream()))


def mmq_q4k_q8_fp32out(w, m, k, q, ds, n, out):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q4k"), m, k, q, n * k, ds, n, out, n * m * 4)
    _check("mmq_q4k_q8_fp32out", load_library().mmq_q4k_q8_fp32out(
        _ptr(w), m, k, _ptr(q), _ptr(ds), n, _ptr(out), _stream()))


def mmq_q4k_q8_f16out(w, m, k, q, ds, n, out):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q4k"), m, k, q, n * k, ds, n, out, n * m * 2)
    _check("mmq_q4k_q8_f16out", load_library().mmq_q4k_q8_f16out(
        _ptr(w), m, k, _ptr(q), _ptr(ds), n, _ptr(out), _stream()))


def mmq_q4k_q8_fold(w, m, k, q, ds, n, out, out_f16, kernel):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q4k"), m, k, q, n * k, ds, n, out, n * m * (2 if out_f16 else 4))
    _check("mmq_q4k_q8_fold", load_library().mmq_q4k_q8_fold(
        _ptr(w), m, k, _ptr(q), _ptr(ds), n, _ptr(out), int(out_f16), int(kernel), _stream()))


def q4k_repack(w, m, k, wr):
    if m >= 0 and k > 0 and k % 256 == 0:
        _fits(w, _w_bytes(m, k, "q4k"), "w")
        _fits(wr, _w_bytes(m, k, "repacked"), "wr")
        _same_device(w, wr)
    _check("q4k_repack", load_library().q4k_repack(_ptr(w), m, k, _ptr(wr), _stream()))


def mmq_q4kr_q8_fp32out(wr, m, k, q, ds, n, out):
    if _sized(m, k, n):
        _check_fold_args(wr, _w_bytes(m, k, "repacked"), m, k, q, n * k, ds, n, out, n * m * 4)
    _check("mmq_q4kr_q8_fp32out", load_library().mmq_q4kr_q8_fp32out(
        _ptr(wr), m, k, _ptr(q), _ptr(ds), n, _ptr(out), _stream()))


def mmq_q4k_q8t_fp32out(w, m, k, qt, ds, n, out):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q4k"), m, k, qt, tiles_elems(n, k) * 2, ds, n, out, n * m * 4)
    _check("mmq_q4k_q8t_fp32out", load_library().mmq_q4k_q8t_fp32out(
        _ptr(w), m, k, _ptr(qt), _ptr(ds), n, _ptr(out), _stream()))


def mmq_q4kr_q8t_fp32out(wr, m, k, qt, ds, n, out):
    if _sized(m, k, n):
        _check_fold_args(wr, _w_bytes(m, k, "repacked"), m, k, qt, tiles_elems(n, k) * 2, ds, n, out, n * m * 4)
    _check("mmq_q4kr_q8t_fp32out", load_library().mmq_q4kr_q8t_fp32out(
        _ptr(wr), m, k, _ptr(qt), _ptr(ds), n, _ptr(out), _stream()))


def mmq_q6k_q8t_fp32out(w, m, k, qt, ds, n, out):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q6k"), m, k, qt, tiles_elems(n, k) * 2, ds, n, out, n * m * 4)
    _check("mmq_q6k_q8t_fp32out", load_library().mmq_q6k_q8t_fp32out(
        _ptr(w), m, k, _ptr(qt), _ptr(ds), n, _ptr(out), _stream()))


def mmq_q6k_q8(w, m, k, q, ds, n, dots):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q6k"), m, k, q, n * k, None, n, dots, n * m * (k // 16) * 4)
        _fits(ds, n * (k // 32) * 4, "ds")
    _check("mmq_q6k_q8", load_library().mmq_q6k_q8(
        _ptr(w), m, k, _ptr(q), _ptr(ds), n, _ptr(dots), _stream()))


def mmq_q6k_q8_fp32out(w, m, k, q, ds, n, out):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q6k"), m, k, q, n * k, ds, n, out, n * m * 4)
    _check("mmq_q6k_q8_fp32out", load_library().mmq_q6k_q8_fp32out(
        _ptr(w), m, k, _ptr(q), _ptr(ds), n, _ptr(out), _stream()))


def mmq_q6k_q8_f16out(w, m, k, q, ds, n, out):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q6k"), m, k, q, n * k, ds, n, out, n * m * 2)
    _check("mmq_q6k_q8_f16out", load_library().mmq_q6k_q8_f16out(
        _ptr(w), m, k, _ptr(q), _ptr(ds), n, _ptr(out), _stream()))


def mmq_q6k_q8_fold(w, m, k, q, ds, n, out, out_f16, kernel):
    if _sized(m, k, n):
        _check_fold_args(w, _w_bytes(m, k, "q6k"), m, k, q, n * k, ds, n, out, n * m * (2 if out_f16 else 4))
    _check("mmq_q6k_q8_fold", load_library().mmq_q6k_q8_fold(
        _ptr(w), m, k, _ptr(q), _ptr(ds), n, _ptr(out), int(out_f16), int(kernel), _stream()))


def mmq_kernel_choice(fmt: int, m: int, k: int, n: int) -> int:
    """The kernel id (KERNEL_*) a fold entry point of format fmt runs for an
    m x k weight and n tokens (host logic only; raises on a bad argument)."""
    r = load_library().mmq_kernel_choice(int(fmt), m, k, n)
    _check("mmq_kernel_choice", r if r < 0 else 0)
    return r


# --------------------------------------------------------- tensor helpers
def _tokens(q, k, name="q"):
    """Token count of a q8 code tensor [n, k] (raises unless its rows are k long)."""
    if q.dim() != 2 or q.shape[1] != k:
        raise ValueError("%s must be [n, %d], got %s" % (name, k, tuple(q.shape)))
    return q.shape[0]


def _scale_words(ds, n, k):
    if tuple(ds.shape) != (n, k // 32):
        raise ValueError("ds must be [%d, %d], got %s" % (n, k // 32, tuple(ds.shape)))


def _out_tensor(out, n, m, dtype, dev):
    if out is None:
        return torch.empty((n, m), dtype=dtype, device=dev)
    _need(out, dtype, "out")
    if tuple(out.shape) != (n, m):
        raise ValueError("out must be [%d, %d], got %s" % (n, m, tuple(out.shape)))
    return out


def _weights(w, m, k, fmt, name="w"):
    _need(w, torch.uint8, name)
    _mmq_sizes(m, k, 0)
    if w.numel() != _w_bytes(m, k, fmt):
        raise ValueError("%s must hold %d bytes for a %d x %d %s matrix, got %d"
                         % (name, _w_bytes(m, k, fmt), m, k, fmt, w.numel()))


def quantize(x: torch.Tensor):
    """x float32 [n, k] -> (q int8 [n, k], ds int32 [n, k/32] holding the uint32 words)."""
    _need(x, torch.float32, "x")
    if x.dim() != 2:
        raise ValueError("x must be [n, k]")
    n, k = x.shape
    q = torch.empty((n, k), dtype=torch.int8, device=x.device)
    ds = torch.empty((n, k // 32 if k % 32 == 0 else 0), dtype=torch.int32, device=x.device)
    q8_quantize_rows(x, n, k, q, ds)
    return q, ds


def tiles_elems(n: int, k: int) -> int:
    """binary16 values in q8_quantize_rows_tiled's output for n tokens of k."""
    return (n + 127) // 128 * 128 * k


def quantize_tiled(x: torch.Tensor):
    """x float32 [n, k] -> (qt int16 [tiles_elems(n, k)] holding the binary16
    operand tiles, ds int32 [n, k/32])."""
    _need(x, torch.float32, "x")
    if x.dim() != 2:
        raise ValueError("x must be [n, k]")
    n, k = x.shape
    qt = torch.empty(tiles_elems(n, k), dtype=torch.int16, device=x.device)
    ds = torch.empty((n, k // 32 if k % 32 == 0 else 0), dtype=torch.int32, device=x.device)
    q8_quantize_rows_tiled(x, n, k, qt, ds)
    return qt, ds


def quantize_silu_mul_tiled(gate: torch.Tensor, up: torch.Tensor):
    """Operand tiles of q8(SiLU(gate) * up): (qt int16 [tiles_elems(n, k)], ds int32 [n, k/32])."""
    _need(gate, torch.float32, "gate")
    _need(up, torch.float32, "up")
    if gate.shape != up.shape or gate.dim() != 2:
        raise ValueError("gate and up must have the same shape [n, k]")
    n, k = gate.shape
    qt = torch.empty(tiles_elems(n, k), dtype=torch.int16, device=gate.device)
    ds = torch.empty((n, k // 32 if k % 32 == 0 else 0), dtype=torch.int32, device=gate.device)
    q8_quantize_silu_mul_tiled(gate, up, n, k, qt, ds)
    return qt, ds


def quantize_silu_mul(gate: torch.Tensor, up: torch.Tensor):
    """q8 of SiLU(gate) * up: (q int8 [n, k], ds int32 [n, k/32])."""
    _need(gate, torch.float32, "gate")
    _need(up, torch.float32, "up")
    if gate.shape != up.shape or gate.dim() != 2:
        raise ValueError("gate and up must have the same shape [n, k]")
    n, k = gate.shape
    q = torch.empty((n, k), dtype=torch.int8, device=gate.device)
    ds = torch.empty((n, k // 32 if k % 32 == 0 else 0), dtype=torch.int32, device=gate.device)
    q8_quantize_silu_mul(gate, up, n, k, q, ds)
    return q, ds


def blockdots(w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds=None):
    """Exact int32 block dots [n, m, k/32]."""
    _weights(w, m, k, "q4k")
    _need(q, torch.int8, "q")
    n = _tokens(q, k)
    dots = torch.empty((n, m, k // 32), dtype=torch.int32, device=q.device)
    mmq_q4k_q8(w, m, k, q, ds, n, dots)
    return dots


def _fold(w, m, k, q, ds, out, fmt, out_dtype, call):
    _weights(w, m, k, fmt)
    _need(q, torch.int8, "q")
    _need(ds, torch.int32, "ds")
    n = _tokens(q, k)
    _scale_words(ds, n, k)
    out = _out_tensor(out, n, m, out_dtype, q.device)
    call(w, m, k, q, ds, n, out)
    return out


def fp32(w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds: torch.Tensor, out=None):
    """Two-term-fold output float32 [n, m]."""
    return _fold(w, m, k, q, ds, out, "q4k", torch.float32, mmq_q4k_q8_fp32out)


def fp16(w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds: torch.Tensor, out=None):
    """Two-term-fold output as binary16 [n, m] (the float32 result, rounded to nearest-even)."""
    return _fold(w, m, k, q, ds, out, "q4k", torch.float16, mmq_q4k_q8_f16out)


def fold_kernel(w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds: torch.Tensor, kernel: int,
                f16: bool = False, out=None):
    """The q4_K fold on a named kernel (KERNEL_*): float32 or binary16 [n, m]."""
    return _fold(w, m, k, q, ds, out, "q4k", torch.float16 if f16 else torch.float32,
                 lambda *a: mmq_q4k_q8_fold(*a, int(f16), kernel))


def q6k_dots(w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds=None):
    """Exact int32 q6_K group dots [n, m, k/16]."""
    _weights(w, m, k, "q6k")
    _need(q, torch.int8, "q")
    n = _tokens(q, k)
    dots = torch.empty((n, m, k // 16), dtype=torch.int32, device=q.device)
    mmq_q6k_q8(w, m, k, q, ds, n, dots)
    return dots


def q6k_fp32(w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds: torch.Tensor, out=None):
    """q6_K output float32 [n, m]."""
    return _fold(w, m, k, q, ds, out, "q6k", torch.float32, mmq_q6k_q8_fp32out)


def q6k_fp16(w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds: torch.Tensor, out=None):
    """q6_K output as binary16 [n, m] (the float32 result, rounded to nearest-even)."""
    return _fold(w, m, k, q, ds, out, "q6k", torch.float16, mmq_q6k_q8_f16out)


def q6k_fold_kernel(w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds: torch.Tensor, kernel: int,
                    f16: bool = False, out=None):
    """The q6_K fold on a named kernel (KERNEL_*): float32 or binary16 [n, m]."""
    return _fold(w, m, k, q, ds, out, "q6k", torch.float16 if f16 else torch.float32,
                 lambda *a: mmq_q6k_q8_fold(*a, int(f16), kernel))


def _tiles_fold(w, m, k, qt, ds, out, fmt, call):
    _weights(w, m, k, fmt)
    _need(qt, torch.int16, "qt")
    _need(ds, torch.int32, "ds")
    if ds.dim() != 2:
        raise ValueError("ds must be [n, k/32]")
    n = ds.shape[0]
    _scale_words(ds, n, k)
    if qt.numel() != tiles_elems(n, k):
        raise ValueError("qt must hold tiles_elems(%d, %d) = %d values, got %d"
                         % (n, k, tiles_elems(n, k), qt.numel()))
    out = _out_tensor(out, n, m, torch.float32, ds.device)
    call(w, m, k, qt, ds, n, out)
    return out


def fp32_tiles(w: torch.Tensor, m: int, k: int, qt: torch.Tensor, ds: torch.Tensor, out=None,
               repacked: bool = False):
    """The fold on q8 operand tiles (from quantize_tiled): float32 [n, m]; w is
    q4_K rows, or q4k_repack records with repacked=True."""
    return _tiles_fold(w, m, k, qt, ds, out, "repacked" if repacked else "q4k",
                       mmq_q4kr_q8t_fp32out if repacked else mmq_q4k_q8t_fp32out)


def q6k_fp32_tiles(w: torch.Tensor, m: int, k: int, qt: torch.Tensor, ds: torch.Tensor, out=None):
    """The q6_K fold on q8 operand tiles (from quantize_tiled): float32 [n, m]."""
    return _tiles_fold(w, m, k, qt, ds, out, "q6k", mmq_q6k_q8t_fp32out)


def repack_bytes(m: int, k: int) -> int:
    """Size of q4k_repack's output for an m x k matrix."""
    return _w_bytes(m, k, "repacked")


def repack(w: torch.Tensor, m: int, k: int):
    """Load-time repack of q4_K weights: uint8 tensor of repack_bytes(m, k)."""
    _weights(w, m, k, "q4k")
    wr = torch.empty(repack_bytes(m, k), dtype=torch.uint8, device=w.device)
    q4k_repack(w, m, k, wr)
    return wr


def fp32_repacked(wr: torch.Tensor, m: int, k: int, q: torch.Tensor, ds: torch.Tensor, out=None):
    """mmq_q4k_q8_fp32out on repacked weights: float32 [n, m]."""
    return _fold(wr, m, k, q, ds, out, "repacked", torch.float32, mmq_q4kr_q8_fp32out)


# ------------------------------------------------- epilogue, experts, norm
def _run(fn: str, dev, *args):
    """Call the library with the current stream of dev, dev being the current
    device meanwhile (a launch goes to the current one)."""
    call, i = getattr(load_library(), fn), dev.index
    if i == torch.cuda.current_device():
        rc = call(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            rc = call(*args, torch._C._cuda_getCurrentRawStream(i))
    if rc != 0:
        _check(fn, rc)


def _on_one(dev, *ts):
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on one device, got %s and %s" % (dev, t.device))


def _rows(t, dtypes, n: int, k: int, name: str) -> int:
    """The row stride of a [n, k] tensor with contiguous rows, 0 for n < 2."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or not t.is_cuda:
        raise TypeError("%s must be a %s tensor on a HIP device" % (name, " or ".join(str(d) for d in dtypes)))
    if t.shape != (n, k):
        raise ValueError("%s must be [%d, %d], got %s" % (name, n, k, tuple(t.shape)))
    rows, columns = t.stride()
    if columns != 1 and k > 1:
        raise ValueError("%s must have contiguous rows" % name)
    if n < 2:
        return 0
    if rows < k:
        raise ValueError("%s has a row stride below %d" % (name, k))
    return rows


def _vector(t, k: int, name: str):
    _need(t, torch.float32, name)
    if tuple(t.shape) != (k,):
        raise ValueError("%s must be [%d], got %s" % (name, k, tuple(t.shape)))


_F32, _FLOATS = (torch.float32,), (torch.float32, torch.float16)


def _addr(t):
    return None if t is None else t.data_ptr()


def _norm_args(x, weight, eps, y, y_weight, gate, residual_scale, r, h):
    """(Norm, n, k, r, tensors) of a norm call; r: the new residual stream."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [n, k]")
    n, k = x.shape
    a = Norm()
    a.x_stride = _rows(x, _F32, n, k, "x")
    _vector(weight, k, "weight")
    if y is None:
        if y_weight is not None or gate is not None or r is not None or residual_scale != 1.0:
            raise ValueError("y_weight, gate, r and residual_scale need y")
        r = x
    else:
        a.y_stride = _rows(y, _FLOATS, n, k, "y")
        a.y_f16 = y.dtype == torch.float16
        if y_weight is not None:
            _vector(y_weight, k, "y_weight")
        if gate is not None:
            if isinstance(gate, torch.Tensor) and gate.dim() == 1:
                _vector(gate, k, "gate")
            else:
                a.gate_stride = _rows(gate, _F32, n, k, "gate")
        if r is None:
            r = torch.empty((n, k), dtype=torch.float32, device=x.device)
        a.r_stride = _rows(r, _F32, n, k, "r")
        a.r = r.data_ptr()
    if h is not None:
        _need(h, torch.float32, "h")
        if tuple(h.shape) != (n, k):
            raise ValueError("h must be [%d, %d], got %s" % (n, k, tuple(h.shape)))
    _on_one(x.device, weight, y, y_weight, gate, r, h)
    a.x, a.y, a.y_weight, a.gate = _addr(x), _addr(y), _addr(y_weight), _addr(gate)
    a.weight, a.h, a.residual_scale, a.eps = _addr(weight), _addr(h), residual_scale, eps
    return a, n, k, r


def quantize_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, y=None, y_weight=None, gate=None,
                  residual_scale: float = 1.0, r=None, h=None):
    """q8 of the normed residual stream (q8_quantize_norm): (q int8 [n, k],
    ds int32 [n, k/32], r).  x float32 [n, k]; y float32 or binary16 [n, k];
    gate [k] or [n, k]; r: where the new stream goes (x itself is fine), x
    without y; h: a float32 [n, k] that gets the normed values too.  A token
    with a NaN or an infinity gets NaN scales, and its products are NaN."""
    a, n, k, r = _norm_args(x, weight, eps, y, y_weight, gate, residual_scale, r, h)
    q = torch.empty((n, k), dtype=torch.int8, device=x.device)
    ds = torch.empty((n, k // 32), dtype=torch.int32, device=x.device)
    _run("q8_quantize_norm", x.device, a, n, k, q.data_ptr(), ds.data_ptr())
    return q, ds, r


def quantize_norm_tiled(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, y=None, y_weight=None, gate=None,
                        residual_scale: float = 1.0, r=None, h=None):
    """quantize_norm with the codes as operand tiles: (qt int16
    [tiles_elems(n, k)], ds int32 [n, k/32], r)."""
    a, n, k, r = _norm_args(x, weight, eps, y, y_weight, gate, residual_scale, r, h)
    qt = torch.empty(tiles_elems(n, k), dtype=torch.int16, device=x.device)
    ds = torch.empty((n, k // 32), dtype=torch.int32, device=x.device)
    _run("q8_quantize_norm_tiled", x.device, a, n, k, qt.data_ptr(), ds.data_ptr())
    return qt, ds, r


def norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, y=None, y_weight=None, gate=None,
         residual_scale: float = 1.0, r=None, h=None):
    """The normed residual stream in float32 (residual_norm): (h [n, k], r);
    arguments as for quantize_norm."""
    if h is None:
        h = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    a, n, k, r = _norm_args(x, weight, eps, y, y_weight, gate, residual_scale, r, h)
    _run("residual_norm", x.device, a, n, k)
    return h, r


def _epilogue(bias, bias_shape, activation, residual, n, m, out, f16, dev):
    """(Epilogue, out) of a call with n rows of m outputs."""
    a = Epilogue()
    if bias is not None:
        _need(bias, torch.float32, "bias")
        if tuple(bias.shape) != bias_shape:
            raise ValueError("bias must be %s, got %s" % (list(bias_shape), tuple(bias.shape)))
        a.bias = bias.data_ptr()
    if residual is not None:
        a.residual_stride = _rows(residual, _FLOATS, n, m, "residual")
        a.residual_f16 = residual.dtype == torch.float16
        a.residual = residual.data_ptr()
    dtype = torch.float16 if f16 else torch.float32
    if out is None:
        out = torch.empty((n, m), dtype=dtype, device=dev)
    a.out_stride = _rows(out, (dtype,), n, m, "out")
    a.out_f16, a.activation = f16, activation
    return a, out


def fold_epilogue(fmt: int, w: torch.Tensor, m: int, k: int, q: torch.Tensor, ds: torch.Tensor, bias=None,
                  activation: int = ACT_NONE, residual=None, out=None, f16: bool = False):
    """act(fold + bias) + residual of a fold entry point (mmq_fold_epilogue):
    float32 or binary16 [n, m].  fmt: FORMAT_*, q its int8 codes or operand
    tiles; residual and out may have a row stride, and be the same tensor."""
    if fmt not in _FORMAT_NAMES:
        raise ValueError("unknown format %r" % (fmt,))
    _weights(w, m, k, _FORMAT_NAMES[fmt])
    _need(ds, torch.int32, "ds")
    if fmt in _TILE_FORMATS:
        _need(q, torch.int16, "q")
        if ds.dim() != 2:
            raise ValueError("ds must be [n, k/32]")
        n = ds.shape[0]
        if q.numel() != tiles_elems(n, k):
            raise ValueError("q must hold tiles_elems(%d, %d) = %d values, got %d"
                             % (n, k, tiles_elems(n, k), q.numel()))
    else:
        _need(q, torch.int8, "q")
        n = _tokens(q, k)
    _scale_words(ds, n, k)
    a, out = _epilogue(bias, (m,), activation, residual, n, m, out, f16, q.device)
    _on_one(q.device, w, ds, bias, residual, out)
    _run("mmq_fold_epilogue", q.device, fmt, w.data_ptr(), m, k, q.data_ptr(), ds.data_ptr(), n, a, out.data_ptr())
    return out


def fold_grouped(fmt: int, w: torch.Tensor, experts: int, m: int, k: int, q: torch.Tensor, ds: torch.Tensor,
                 offsets: torch.Tensor, rows=None, bias=None, activation: int = ACT_NONE, residual=None, out=None,
                 f16: bool = False):
    """Matrix products grouped by expert (mmq_fold_grouped): float32 or
    binary16 [slots, m].  w: experts matrices of m x k (FORMAT_Q4K or
    FORMAT_Q6K); offsets int32 [experts + 1]; rows int32 [slots], the row of q
    of each slot, or None (slot s takes row s); bias [experts, m].  slots is
    the length of rows, or the rows of q without it, and no more than out has;
    rows of out that belong to no expert are left as they were (uninitialised
    in a new tensor).  residual [slots, m] may be out."""
    if fmt not in (FORMAT_Q4K, FORMAT_Q6K):
        raise ValueError("grouped products take FORMAT_Q4K or FORMAT_Q6K, got %r" % (fmt,))
    if experts < 1:
        raise ValueError("experts must be positive, got %d" % experts)
    _mmq_sizes(m, k, 0)
    _weights(w, experts * m, k, _FORMAT_NAMES[fmt])
    _need(q, torch.int8, "q")
    _need(ds, torch.int32, "ds")
    tokens = _tokens(q, k)
    _scale_words(ds, tokens, k)
    _need(offsets, torch.int32, "offsets")
    if tuple(offsets.shape) != (experts + 1,):
        raise ValueError("offsets must be [%d], got %s" % (experts + 1, tuple(offsets.shape)))
    if rows is not None:
        _need(rows, torch.int32, "rows")
        if rows.dim() != 1:
            raise ValueError("rows must be [slots]")
    slots = tokens if rows is None else rows.shape[0]
    if out is not None and out.dim() == 2 and out.shape[0] < slots:
        slots = out.shape[0]
    a, out = _epilogue(bias, (experts, m), activation, residual, slots, m, out, f16, q.device)
    _on_one(q.device, w, ds, offsets, rows, bias, residual, out)
    _run("mmq_fold_grouped", q.device, fmt, w.data_ptr(), experts, m, k, q.data_ptr(), ds.data_ptr(), tokens,
         _addr(rows), offsets.data_ptr(), slots, a, out.data_ptr())
    return out


def route(logits: torch.Tensor, top: int, normalize: bool = True, scale: float = 1.0) -> Routing:
    """The router of fold_grouped (moe_route) on float32 scores [n, experts]:
    top experts of each token, their weights, and the slots of the grouped
    products."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be [n, experts]")
    n, experts = logits.shape
    stride = _rows(logits, _F32, n, experts, "logits")
    if not 1 <= top <= min(experts, 64):
        raise ValueError("top must be 1 .. min(experts, 64), got %d of %d" % (top, experts))
    dev = logits.device
    ids = torch.empty((n, top), dtype=torch.int32, device=dev)
    weights = torch.empty((n, top), dtype=torch.float32, device=dev)
    slot = torch.empty((n, top), dtype=torch.int32, device=dev)
    rows = torch.empty(n * top, dtype=torch.int32, device=dev)
    offsets = (torch.empty if n else torch.zeros)(experts + 1, dtype=torch.int32, device=dev)
    _run("moe_route", dev, logits.data_ptr(), n, experts, stride, top, normalize, scale, ids.data_ptr(),
         weights.data_ptr(), slot.data_ptr(), rows.data_ptr(), offsets.data_ptr())
    return Routing(ids, weights, slot, rows, offsets)


def combine(y: torch.Tensor, slot: torch.Tensor, weights: torch.Tensor, residual=None, out=None):
    """The experts' outputs back in token order (moe_combine): float32 [n, m],
    residual + sum_j weights[:, j] * y[slot[:, j]].  y float32 or binary16
    [slots, m]; residual may be out."""
    if not isinstance(y, torch.Tensor) or y.dtype not in _FLOATS:
        raise TypeError("y must be a float32 or binary16 tensor")
    _need(y, y.dtype, "y")
    _need(slot, torch.int32, "slot")
    _need(weights, torch.float32, "weights")
    if y.dim() != 2 or slot.dim() != 2 or slot.shape != weights.shape:
        raise ValueError("need y [slots, m] and slot, weights [n, top], got %s, %s, %s"
                         % (tuple(y.shape), tuple(slot.shape), tuple(weights.shape)))
    (n, top), (slots, m) = slot.shape, y.shape
    if residual is not None:
        _need(residual, torch.float32, "residual")
        if tuple(residual.shape) != (n, m):
            raise ValueError("residual must be [%d, %d], got %s" % (n, m, tuple(residual.shape)))
    out = _out_tensor(out, n, m, torch.float32, y.device)
    _on_one(y.device, slot, weights, residual, out)
    _run("moe_combine", y.device, y.data_ptr(), y.dtype == torch.float16, slots, m, slot.data_ptr(),
         weights.data_ptr(), n, top, _addr(residual), out.data_ptr())
    return out


# ------------------------------------------------- positions, cache, attention
def _rope_args(rope, n: int, dev):
    """RopeArgs of a Rope for n rows."""
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope, got %s" % type(rope).__name__)
    p, freq, axis, adjacent, scale = rope
    _need(freq, torch.float32, "freq")
    if freq.dim() != 1:
        raise ValueError("freq must be [pairs], got %s" % (tuple(freq.shape),))
    if not isinstance(p, torch.Tensor) or not 1 <= p.dim() <= 2:
        raise TypeError("positions must be an int32 tensor [n] or [n, axes] on a HIP device")
    if p.shape[0] != n:
        raise ValueError("positions must have %d rows, got %s" % (n, tuple(p.shape)))
    if p.dim() == 1:
        _need(p, torch.int32, "positions")
        axes, stride = 1, 1
    else:
        axes = p.shape[1]
        stride = _rows(p, (torch.int32,), n, axes, "positions")
    if axis is not None:
        _need(axis, torch.int32, "axis")
        if axis.shape != freq.shape:
            raise ValueError("axis must be [%d], got %s" % (freq.shape[0], tuple(axis.shape)))
    _on_one(dev, p, freq, axis)
    return RopeArgs(p.data_ptr(), freq.data_ptr(), _addr(axis), stride, axes, freq.shape[0], adjacent, scale)


def _matrix(t, name: str, columns=None):
    """(rows, columns) of a float32 or binary16 matrix."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _FLOATS or t.dim() != 2:
        raise TypeError("%s must be a float32 or binary16 matrix" % name)
    if columns is not None and t.shape[1] != columns:
        raise ValueError("%s must have %d columns, got %s" % (name, columns, tuple(t.shape)))
    return t.shape


def rope(x: torch.Tensor, heads: int, rope: Rope, out=None) -> torch.Tensor:
    """Rotary positions on rows of heads (rope_rows): x float32 or binary16
    [n, heads * head_dim], out alike (x itself is fine)."""
    n, columns = _matrix(x, "x")
    if heads < 1 or columns % heads:
        raise ValueError("x has %d columns, not a multiple of %d heads" % (columns, heads))
    if out is None:
        out = torch.empty((n, columns), dtype=x.dtype, device=x.device)
    xs, outs = _rows(x, _FLOATS, n, columns, "x"), _rows(out, (x.dtype,), n, columns, "out")
    a = _rope_args(rope, n, x.device)
    _on_one(x.device, out)
    _run("rope_rows", x.device, a, x.data_ptr(), xs, x.dtype == torch.float16, n, heads, columns // heads,
         out.data_ptr(), outs)
    return out


def _cache_args(pages: int, heads: int, head_dim: int, page: int, fmt: int) -> CacheArgs:
    a = CacheArgs()
    a.pages, a.heads, a.head_dim, a.page, a.format = pages, heads, head_dim, page, fmt
    return a


def cache_bytes(pages: int, heads: int, head_dim: int, page: int = 64, fmt: int = KV_Q8) -> int:
    """Bytes of a cache (kv_cache_bytes)."""
    n = ctypes.c_int64()
    _check("kv_cache_bytes", load_library().kv_cache_bytes(_cache_args(pages, heads, head_dim, page, fmt), n))
    return n.value


def new_cache(pages: int, heads: int, head_dim: int, page: int = 64, fmt: int = KV_Q8, device="cuda") -> KVCache:
    """A cache of `pages` pages of `page` tokens (not cleared: what is not
    written is not read into any result)."""
    record = cache_bytes(pages, heads, head_dim, page, fmt) // (pages * heads)
    return KVCache(torch.empty((pages, heads, record), dtype=torch.uint8, device=device), head_dim, page, fmt)


def _kv_args(cache, plan):
    """(CacheArgs, PlanArgs, kv heads) of a call."""
    if not isinstance(cache, KVCache) or not isinstance(plan, KVPlan):
        raise TypeError("need a KVCache and a KVPlan")
    data, head_dim, page, fmt = cache
    table, lengths, offsets = plan
    _need(data, torch.uint8, "data")
    if data.dim() != 3:
        raise ValueError("data must be [pages, heads, bytes], got %s" % (tuple(data.shape),))
    pages, heads, record = data.shape
    if record != 2 * page * ((head_dim // 2 if fmt == KV_Q4 else head_dim) + head_dim // 16):
        raise ValueError("records of %d bytes do not hold pages of %d tokens of %d values" % (record, page, head_dim))
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [seqs, width]")
    seqs, width = table.shape
    stride = _rows(table, (torch.int32,), seqs, width, "table")
    _need(lengths, torch.int32, "lengths")
    if lengths.shape != (seqs,):
        raise ValueError("lengths must be [%d], got %s" % (seqs, tuple(lengths.shape)))
    at = None
    if offsets is not None:
        _need(offsets, torch.int32, "offsets")
        if offsets.shape != (seqs + 1,):
            raise ValueError("offsets must be [%d], got %s" % (seqs + 1, tuple(offsets.shape)))
        at = offsets.data_ptr()
    _on_one(data.device, table, lengths, offsets)
    return (CacheArgs(data.data_ptr(), pages, heads, head_dim, page, fmt),
            PlanArgs(table.data_ptr(), lengths.data_ptr(), at, seqs, width, stride), heads)


def kv_write(cache: KVCache, plan: KVPlan, k: torch.Tensor, v: torch.Tensor, rope: Optional[Rope] = None) -> None:
    """New tokens' keys and values into the cache (kv_write), the keys rotated
    first with rope: k, v float32 or binary16 [n, kv heads * head_dim]."""
    c, p, heads = _kv_args(cache, plan)
    columns = heads * cache.head_dim
    n, _ = _matrix(k, "k", columns)
    ks, vs = _rows(k, _FLOATS, n, columns, "k"), _rows(v, (k.dtype,), n, columns, "v")
    dev = cache.data.device
    a = None if rope is None else _rope_args(rope, n, dev)
    _on_one(dev, k, v)
    _run("kv_write", dev, c, p, a, k.data_ptr(), v.data_ptr(), k.dtype == torch.float16, n, ks, vs)


def kv_read(cache: KVCache, plan: KVPlan, n: int, f16: bool = True, k=None, v=None):
    """n rows read back (kv_read): (k, v), binary16 or float32
    [n, kv heads * head_dim].  Rows that belong to no sequence are left as they
    were (uninitialised in new tensors)."""
    c, p, heads = _kv_args(cache, plan)
    dtype, dev, columns = torch.float16 if f16 else torch.float32, cache.data.device, heads * cache.head_dim
    if n < 0:
        raise ValueError("n must not be negative, got %d" % n)
    if k is None:
        k = torch.empty((n, columns), dtype=dtype, device=dev)
    if v is None:
        v = torch.empty((n, columns), dtype=dtype, device=dev)
    ks, vs = _rows(k, (dtype,), n, columns, "k"), _rows(v, (dtype,), n, columns, "v")
    _on_one(dev, k, v)
    _run("kv_read", dev, c, p, k.data_ptr(), v.data_ptr(), f16, n, ks, vs)
    return k, v


def kv_attend(cache: KVCache, plan: KVPlan, q: torch.Tensor, heads: int, scale: Optional[float] = None,
              window: int = 0, most: Optional[int] = None, out=None, f16: Optional[bool] = None, lse: bool = False):
    """Causal attention of new tokens over the cache, which holds them already
    (kv_attend): q float32 or binary16 [n, heads * head_dim], out alike, or as
    f16 says.  scale: 1 / sqrt(head_dim) by default; window: how many tokens a
    row sees, 0 for all; most: an upper bound of a sequence's rows (1 without
    offsets, else n, which costs time where sequences have few of them: 125 us
    for 63 decoding sequences of 4000 tokens, 210 by default).  Returns out, or (out, lse float32 [n, heads]) with lse.
    Rows that belong to no sequence are left as they were."""
    c, p, _ = _kv_args(cache, plan)
    columns, dev = heads * cache.head_dim, cache.data.device
    n, _ = _matrix(q, "q", columns)
    q_stride = _rows(q, _FLOATS, n, columns, "q")
    if not 0 <= window < 1 << 31:
        raise ValueError("window must be 0 .. 2^31 - 1, got %d" % window)
    if f16 is None:
        f16 = (q if out is None else out).dtype == torch.float16
    dtype = torch.float16 if f16 else torch.float32
    if out is None:
        out = torch.empty((n, columns), dtype=dtype, device=dev)
    out_stride = _rows(out, (dtype,), n, columns, "out")
    sums = torch.empty((n, heads), dtype=torch.float32, device=dev) if lse else None
    _on_one(dev, q, out)
    if most is None:
        most = max(1, n if plan.offsets is not None else 1)
    a = QueryArgs(q.data_ptr(), out.data_ptr(), _addr(sums), q_stride, out_stride, n, most, heads,
                  q.dtype == torch.float16, f16, window, cache.head_dim ** -0.5 if scale is None else scale)
    need = ctypes.c_int64()
    rc = load_library().kv_attend_workspace(c, p, a, need)
    if rc != 0:
        _check("kv_attend_workspace", rc)
    space = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
    _run("kv_attend", dev, c, p, a, _addr(space), need.value)
    return (out, sums) if lse else out
