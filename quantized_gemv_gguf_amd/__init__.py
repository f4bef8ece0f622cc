"""Python binding of libqgemv.so (include/qgemv.h): batch-1 dequant-GEMV over
GGUF block-quantized weights (Q8_0, Q4_0, MXFP4, Q4_K, Q6_K) on MI355X.

The functions carry the C names and do argument marshalling only: torch
tensors are turned into raw pointers and sizes, the caller's torch stream into
a ``hipStream_t``, and a negative status into :class:`QgemvError`.  Every step
of the computation runs in the library's HIP kernels; there is no other path.
If ``libqgemv.so`` is missing, importing works but every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Sequence

Q8_0, Q4_0, MXFP4, Q4_K, Q6_K = 1, 2, 3, 4, 5
F32, F16, BF16 = 32, 33, 34  # float element types of a qg_tensor (qgemv_mx.h)
FORMATS = {"q8_0": Q8_0, "q4_0": Q4_0, "mxfp4": MXFP4, "q4_k": Q4_K, "q6_k": Q6_K}
MAX_WINDOWS = 64
MAX_K = 49152
CHAIN_MAX_K = 24576
MAX_EXPERTS = 1024
MAX_SEQS, MAX_HEADS, MAX_HEAD_DIM, MAX_POOL_PAGES = 4096, 1024, 256, 1 << 22
ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3
IN_X, IN_RMS, IN_GELU_RMS, IN_SILU_MUL = 0, 1, 2, 3
OUT_Y, OUT_GELU = 0, 1

QG_OK = 0
STATUS = {
    -1: "QG_E_NULL", -2: "QG_E_FMT", -3: "QG_E_SHAPE", -4: "QG_E_RANGE", -5: "QG_E_SIZE",
    -6: "QG_E_ARG", -7: "QG_E_NOT_PINNED", -8: "QG_E_CAPACITY", -9: "QG_E_BARRIER", -100: "QG_E_HIP",
}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemv.so")

_i32, _i64, _f64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p


class QgemvError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        self.name = STATUS.get(status, str(status))
        msg = f"{where}: {self.name} ({status})"
        if detail:
            msg += f": {detail}"
        super().__init__(msg)


class qg_matrix(ctypes.Structure):
    _fields_ = [("data", _vp), ("fmt", _i32), ("reserved", _i32), ("n_rows", _i64), ("k", _i64),
                ("n_bytes", _i64)]


class qg_window(ctypes.Structure):
    _fields_ = [("data", _vp), ("n_rows", _i64), ("row_start", _i64), ("row_end", _i64),
                ("x", _vp), ("y", _vp)]


class qg_plan_step(ctypes.Structure):
    _fields_ = [("op", _i32), ("fmt", _i32), ("k", _i64), ("first_win", _i32), ("n_win", _i32),
                ("block_rows", _i64), ("a", _vp), ("b", _vp), ("out", _vp), ("n", _i64), ("stride", _i64),
                ("n_sel", _i32), ("reserved", _i32)]


class qg_chain_window(ctypes.Structure):
    _fields_ = [("data", _vp), ("n_rows", _i64), ("row_start", _i64), ("row_end", _i64),
                ("x", _vp), ("x2", _vp), ("y", _vp)]


class qg_chain_step(ctypes.Structure):
    _fields_ = [("k", _i64), ("first_win", _i32), ("n_win", _i32), ("in_op", _i32), ("eps", ctypes.c_float)]


class qg_tensor(ctypes.Structure):
    _fields_ = [("data", _vp), ("type", _i32), ("reserved", _i32), ("n_rows", _i64), ("n_cols", _i64),
                ("stride", _i64)]


class qg_heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("type", _i32), ("reserved", _i32), ("n_tok", _i64), ("n_head", _i32),
                ("head_dim", _i32), ("tok_stride", _i64), ("head_stride", _i64)]


class qg_rope(ctypes.Structure):
    _fields_ = [("freqs", _vp), ("n_rot", _i32), ("interleaved", _i32), ("mscale", ctypes.c_double)]


class qg_kv_cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("type", _i32), ("page_size", _i32), ("n_layer", _i32), ("n_head", _i32),
                ("head_dim", _i32), ("reserved", _i32), ("n_pages", _i64), ("layer_stride", _i64),
                ("page_stride", _i64), ("head_stride", _i64), ("slot_stride", _i64)]


class qg_kv_seqs(ctypes.Structure):
    _fields_ = [("starts", _vp), ("lens", _vp), ("tables", _vp), ("n_seq", _i32), ("reserved", _i32),
                ("max_pages", _i64)]


class qg_kv_pool(ctypes.Structure):
    _fields_ = [("tables", _vp), ("lens", _vp), ("refs", _vp), ("used", _vp), ("n_seq", _i32), ("page_size", _i32),
                ("max_pages", _i64), ("n_pages", _i64), ("work", _vp), ("work_bytes", _i64)]


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built (run __graft_entry__.build() or "
                           "python quantized_gemv_gguf_amd/build.py); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    sigs = {
        "qgemv_block_bytes": ([_i32], _i64),
        "qgemv_block_weights": ([_i32], _i64),
        "qgemv_weight_bytes": ([_i32, _i64, _i64], _i64),
        "qgemv_rows": ([P(qg_matrix), _i64, _i64, _vp, _vp, _i64, _vp], ctypes.c_int),
        "qgemv_windows": ([_i32, _i64, P(qg_window), _i32, _i64, _vp], ctypes.c_int),
        "qgemv_rows_batch": ([P(qg_matrix), _i64, _i64, _vp, _i64, _i32, _vp, _i64, _i64, _vp], ctypes.c_int),
        "qgemv_rows_mfma": ([P(qg_matrix), _i64, _i64, _vp, _i64, _i32, _vp, _i64, _vp], ctypes.c_int),
        "qgemv_expert_windows_op": ([P(qg_matrix), _i32, _i64, P(_i32), _i32, _vp, _vp, _i64, _i32, ctypes.c_float,
                                     _i32, _vp, _i64, _vp], ctypes.c_int),
        "qgemv_combine": ([_vp, _i64, _i32, _vp, _i64, _vp, _vp], ctypes.c_int),
        "qgemv_rows_swiglu": ([P(qg_matrix), P(qg_matrix), _i64, _i64, _vp, _i32, ctypes.c_float, _vp, _i64, _vp],
                              ctypes.c_int),
        "qgemv_expert_swiglu": ([P(qg_matrix), P(qg_matrix), _i64, P(_i32), _i32, _vp, _i64, _i32, ctypes.c_float,
                                 _vp, _i64, _vp], ctypes.c_int),
        "qgemv_rows_op": ([P(qg_matrix), _i64, _i64, _vp, _vp, _i32, ctypes.c_float, _i32, _vp, _i64, _vp],
                          ctypes.c_int),
        "qgemv_expert_windows": ([P(qg_matrix), _i32, _i64, P(_i32), _i32, _vp, _i64, _vp, _i64, _vp],
                                 ctypes.c_int),
        "qgemv_silu_mul": ([_vp, _vp, _vp, _i64, _vp], ctypes.c_int),
        "qgemv_rms_carry": ([_vp, _vp, _i64, ctypes.c_float, _i32, _vp], ctypes.c_int),
        "qgemv_dequant_rows": ([P(qg_matrix), _i64, _i64, _vp, _vp], ctypes.c_int),
        "qgemv_read_ceiling": ([_vp, _i64, _vp, _vp], ctypes.c_int),
        "qgemv_stream_create": ([_i64, _i32, P(_vp)], ctypes.c_int),
        "qgemv_stream_ring_bytes": ([_vp], _i64),
        "qgemv_stream_rows": ([_vp, P(qg_matrix), _i64, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
        "qgemv_stream_windows": ([_vp, _i32, _i64, P(qg_window), _i32, _i64, _vp], ctypes.c_int),
        "qgemv_stream_destroy": ([_vp], ctypes.c_int),
        "qgemv_stream_plan_create": ([_i64, _i32, P(qg_plan_step), _i32, P(qg_window), _i32, P(_vp)],
                                     ctypes.c_int),
        "qgemv_stream_plan_set_rows": ([_vp, _i32, _i64], ctypes.c_int),
        "qgemv_stream_plan_ring_bytes": ([_vp], _i64),
        "qgemv_stream_plan_run": ([_vp, _vp], ctypes.c_int),
        "qgemv_stream_plan_destroy": ([_vp], ctypes.c_int),
        "qgemv_stream_rows_noalloc": ([P(qg_matrix), _i64, _i64, _i64, _vp, _vp, _vp], ctypes.c_int),
        "qgemv_mapped_rows": ([P(qg_matrix), _i64, _i64, _vp, _vp, _i64, _vp], ctypes.c_int),
        "qgemv_mapped_windows": ([_i32, _i64, P(qg_window), _i32, _i64, _vp], ctypes.c_int),
        "qgemv_chain_create": ([_i32, P(qg_chain_step), _i32, P(qg_chain_window), _i32, P(_vp)], ctypes.c_int),
        "qgemv_chain_run": ([_vp, _vp], ctypes.c_int),
        "qgemv_chain_check": ([_vp], ctypes.c_int),
        "qgemv_chain_set_spin_limit": ([_vp, ctypes.c_uint32], ctypes.c_int),
        "qgemv_chain_grid": ([_vp], _i64),
        "qgemv_chain_destroy": ([_vp], ctypes.c_int),
        "qgemv_mx_quantize": ([P(qg_tensor), P(qg_matrix), _vp], ctypes.c_int),
        "qgemv_mx_dequantize": ([P(qg_matrix), _i64, _i64, P(qg_tensor), _vp], ctypes.c_int),
        "qgemv_rows_mx": ([P(qg_matrix), _i64, _i64, P(qg_tensor), P(qg_tensor), _vp], ctypes.c_int),
        "qgemv_rows_mx_swiglu": ([P(qg_matrix), P(qg_matrix), _i64, _i64, P(qg_tensor), P(qg_tensor), _vp],
                                 ctypes.c_int),
        "qgemv_expert_sort": ([_vp, _i64, _i32, _i64, _vp, _vp, _vp, _vp], ctypes.c_int),
        "qgemv_expert_mx": ([P(qg_matrix), _i64, P(qg_tensor), _vp, _vp, _i32, P(qg_tensor), _vp], ctypes.c_int),
        "qgemv_expert_mx_swiglu": ([P(qg_matrix), P(qg_matrix), _i64, P(qg_tensor), _vp, _vp, _i32, P(qg_tensor),
                                    _vp], ctypes.c_int),
        "qgemv_expert_gather": ([P(qg_tensor), _vp, _i32, P(qg_tensor), _vp], ctypes.c_int),
        "qgemv_expert_combine": ([P(qg_tensor), _vp, _vp, _i32, P(qg_tensor), _vp], ctypes.c_int),
        "qgemv_expert_combine_grad": ([P(qg_tensor), P(qg_tensor), _vp, _vp, _i32, P(qg_tensor), _vp, _vp],
                                      ctypes.c_int),
        "qgemv_rope_freqs": ([_i32, _f64, _i32, _f64, _f64, _f64, _f64, P(_f64), P(_f64)], ctypes.c_int),
        "qgemv_rope": ([_vp, _vp, _vp, _vp, _i32, _vp], ctypes.c_int),
        "qgemv_kv_append": ([_vp, _vp, _vp, _vp, _i32, _vp, _vp,
                             _vp, _vp, _vp], ctypes.c_int),
        "qgemv_kv_attend": ([_vp, _vp, _vp, _i32, _vp, ctypes.c_float, _i32,
                             _i32, _vp, _vp, _vp, _i64, _vp], ctypes.c_int),
        "qgemv_kv_attend_bytes": ([_vp, _vp, _vp], _i64),
        "qgemv_kv_pool_bytes": ([_i64, _i64, _i64], _i64),
        "qgemv_kv_resize": ([_vp, _vp, _vp, _vp], ctypes.c_int),
        "qgemv_kv_fork": ([_vp, _vp, _vp], ctypes.c_int),
        "qgemv_kv_compact": ([_vp, _vp, _vp], ctypes.c_int),
        "qgemv_kv_copy": ([_vp, _vp, _vp, _i64, _vp], ctypes.c_int),
        "qgemv_strerror": ([ctypes.c_int], ctypes.c_char_p),
        "qgemv_last_hip_error": ([], ctypes.c_char_p),
        "qgemv_version": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sigs.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def _check(rc: int, where: str) -> None:
    if rc != QG_OK:
        detail = lib().qgemv_strerror(rc).decode()
        if rc == -100:
            detail += ": " + lib().qgemv_last_hip_error().decode()
        raise QgemvError(rc, where, detail)


# --- marshalling helpers ------------------------------------------------------

def _ptr(t) -> int:
    """Raw address of a tensor (contiguity required), or 0 for None."""
    if t is None:
        return 0
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        # the current stream's handle without a torch.cuda.Stream around it
        # (0.3 us instead of 2.8, a third of a small call's time on the host)
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _f32(t, n: int, name: str):
    import torch
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} values, needs {n}")
    return _ptr(t)


@dataclass
class Matrix:
    """A quantized matrix: ``data`` is a uint8 tensor of the raw blocks (device
    memory for the resident calls, pinned host memory for the streamed ones)."""
    data: object
    fmt: int
    n_rows: int
    k: int

    def c(self) -> qg_matrix:
        return qg_matrix(_ptr(self.data), int(self.fmt), 0, int(self.n_rows), int(self.k),
                         int(self.data.numel() * self.data.element_size()))


@dataclass
class Window:
    """Rows [row_start, row_end) of ``mat`` with input ``x`` (k floats) and
    output ``y`` (row_end - row_start floats)."""
    mat: Matrix
    row_start: int
    row_end: int
    x: object
    y: object

    def c(self) -> qg_window:
        n = self.row_end - self.row_start
        return qg_window(_ptr(self.mat.data), int(self.mat.n_rows), int(self.row_start), int(self.row_end),
                         _f32(self.x, self.mat.k, "x"), _f32(self.y, max(n, 0), "y"))


def _windows(ws: Sequence[Window]):
    if len(ws) == 0:
        return None, 0, None, None
    fmt, k = ws[0].mat.fmt, ws[0].mat.k
    arr = (qg_window * len(ws))(*[w.c() for w in ws])
    return arr, len(ws), fmt, k


# --- entry points ----------------------------------------------------------------

def qgemv_block_bytes(fmt: int) -> int:
    return int(lib().qgemv_block_bytes(fmt))


def qgemv_block_weights(fmt: int) -> int:
    return int(lib().qgemv_block_weights(fmt))


def qgemv_weight_bytes(fmt: int, n_rows: int, k: int) -> int:
    return int(lib().qgemv_weight_bytes(fmt, n_rows, k))


def qgemv_rows(w: Matrix, row_start: int, row_end: int, x, y, block_rows: int = 0, stream=None) -> None:
    m = w.c()
    n = max(row_end - row_start, 0)
    _check(lib().qgemv_rows(ctypes.byref(m), row_start, row_end, _f32(x, w.k, "x"), _f32(y, n, "y"),
                            block_rows, _stream(stream)), "qgemv_rows")


def qgemv_rows_op(w: Matrix, row_start: int, row_end: int, x, y, in_op: int = 0, eps: float = 0.0,
                  out_op: int = 0, x2=None, block_rows: int = 0, stream=None) -> None:
    """As qgemv_rows with a fused input transform (IN_X, IN_RMS, IN_SILU_MUL with ``x2``)
    and output transform (OUT_Y, OUT_GELU)."""
    m = w.c()
    n = max(row_end - row_start, 0)
    x2p = _f32(x2, w.k, "x2") if x2 is not None else None
    _check(lib().qgemv_rows_op(ctypes.byref(m), row_start, row_end, _f32(x, w.k, "x"), x2p, int(in_op),
                               float(eps), int(out_op), _f32(y, n, "y"), block_rows, _stream(stream)),
           "qgemv_rows_op")


def qgemv_rows_batch(w: Matrix, row_start: int, row_end: int, x, y, block_rows: int = 0, stream=None) -> None:
    """y[t] = W[row_start:row_end] . x[t] for every token t: ``x`` is (n_tok, >= k)
    and ``y`` (n_tok, >= row_end - row_start), float32 with unit column stride."""
    m = w.c()
    n = max(row_end - row_start, 0)
    if x.dim() != 2 or y.dim() != 2 or x.shape[0] != y.shape[0]:
        raise ValueError("x and y must be (n_tok, ...) with the same n_tok")
    if x.stride(1) != 1 or y.stride(1) != 1 or x.shape[1] < w.k or y.shape[1] < n:
        raise ValueError("rows of x (k floats) and y (one per output row) must be contiguous")
    nt = x.shape[0]
    _f32(x, 0, "x")
    _f32(y, 0, "y")
    _check(lib().qgemv_rows_batch(ctypes.byref(m), row_start, row_end, _ptr(x), x.stride(0), nt, _ptr(y),
                                  y.stride(0), block_rows, _stream(stream)), "qgemv_rows_batch")


def qgemv_rows_mfma(w: Matrix, row_start: int, row_end: int, x, y, stream=None) -> None:
    """As qgemv_rows_batch on the fp32 matrix cores (every format): y[t]
    within fp32 rounding of W[row_start:row_end] . x[t], not bit-identical to
    the one-token calls."""
    m = w.c()
    n = max(row_end - row_start, 0)
    if x.dim() != 2 or y.dim() != 2 or x.shape[0] != y.shape[0]:
        raise ValueError("x and y must be (n_tok, ...) with the same n_tok")
    if x.stride(1) != 1 or y.stride(1) != 1 or x.shape[1] < w.k or y.shape[1] < n:
        raise ValueError("rows of x (k floats) and y (one per output row) must be contiguous")
    nt = x.shape[0]
    _f32(x, 0, "x")
    _f32(y, 0, "y")
    _check(lib().qgemv_rows_mfma(ctypes.byref(m), row_start, row_end, _ptr(x), x.stride(0), nt, _ptr(y),
                                 y.stride(0), _stream(stream)), "qgemv_rows_mfma")


def qgemv_windows(windows: Sequence[Window], block_rows: int = 0, stream=None, fmt=None, k=None) -> None:
    arr, n, f, kk = _windows(windows)
    f = fmt if f is None else f
    kk = k if kk is None else kk
    _check(lib().qgemv_windows(int(f or Q8_0), int(kk or 32), arr, n, block_rows, _stream(stream)),
           "qgemv_windows")


def qgemv_expert_windows(mats: Sequence[Matrix], n_expert: int, ids, x, x_stride: int, y,
                         block_rows: int = 0, stream=None) -> None:
    ids = [int(i) for i in ids]
    marr = (qg_matrix * len(mats))(*[m.c() for m in mats])
    iarr = (_i32 * max(len(ids), 1))(*ids)
    k = mats[0].k if mats else 32
    out = (mats[0].n_rows // n_expert) if (mats and n_expert > 0) else 0
    xp = _f32(x, k + (len(ids) - 1) * x_stride if ids else 0, "x")
    yp = _f32(y, len(mats) * len(ids) * out, "y")
    _check(lib().qgemv_expert_windows(marr, len(mats), n_expert, iarr, len(ids), xp, x_stride, yp,
                                      block_rows, _stream(stream)), "qgemv_expert_windows")


def qgemv_expert_windows_op(mats: Sequence[Matrix], n_expert: int, ids, x, x_stride: int, y, in_op: int = 0,
                            eps: float = 0.0, out_op: int = 0, x2=None, block_rows: int = 0,
                            stream=None) -> None:
    """As qgemv_expert_windows with qgemv_rows_op's transforms per window (x2
    strided like x, for IN_SILU_MUL)."""
    ids = [int(i) for i in ids]
    marr = (qg_matrix * len(mats))(*[m.c() for m in mats])
    iarr = (_i32 * max(len(ids), 1))(*ids)
    k = mats[0].k if mats else 32
    out = (mats[0].n_rows // n_expert) if (mats and n_expert > 0) else 0
    need = k + (len(ids) - 1) * x_stride if ids else 0
    xp = _f32(x, need, "x")
    x2p = _f32(x2, need, "x2") if x2 is not None else None
    yp = _f32(y, len(mats) * len(ids) * out, "y")
    _check(lib().qgemv_expert_windows_op(marr, len(mats), n_expert, iarr, len(ids), xp, x2p, x_stride, int(in_op),
                                         float(eps), int(out_op), yp, block_rows, _stream(stream)),
           "qgemv_expert_windows_op")


def qgemv_rows_swiglu(gate: Matrix, up: Matrix, row_start: int, row_end: int, x, h, in_op: int = 0,
                      eps: float = 0.0, block_rows: int = 0, stream=None) -> None:
    """h = silu(gate[rows] . x') * (up[rows] . x'), x' = x (IN_X) or rms(x) (IN_RMS)."""
    g, u = gate.c(), up.c()
    n = max(row_end - row_start, 0)
    _check(lib().qgemv_rows_swiglu(ctypes.byref(g), ctypes.byref(u), row_start, row_end, _f32(x, gate.k, "x"),
                                   int(in_op), float(eps), _f32(h, n, "h"), block_rows, _stream(stream)),
           "qgemv_rows_swiglu")


def qgemv_expert_swiglu(gate: Matrix, up: Matrix, n_expert: int, ids, x, x_stride: int, h, in_op: int = 0,
                        eps: float = 0.0, block_rows: int = 0, stream=None) -> None:
    ids = [int(i) for i in ids]
    g, u = gate.c(), up.c()
    iarr = (_i32 * max(len(ids), 1))(*ids)
    out = gate.n_rows // n_expert if n_expert > 0 else 0
    xp = _f32(x, gate.k + (len(ids) - 1) * x_stride if ids else 0, "x")
    _check(lib().qgemv_expert_swiglu(ctypes.byref(g), ctypes.byref(u), n_expert, iarr, len(ids), xp, x_stride,
                                     int(in_op), float(eps), _f32(h, len(ids) * out, "h"), block_rows,
                                     _stream(stream)), "qgemv_expert_swiglu")


def qgemv_combine(y, y_stride: int, n_sel: int, w, n: int, out, stream=None) -> None:
    """out[i] = sum_s w[s] * y[s * y_stride + i] (device tensors)."""
    yp = _f32(y, (n_sel - 1) * y_stride + n if n_sel > 0 else 0, "y")
    wp = _f32(w, n_sel, "w")
    _check(lib().qgemv_combine(yp, y_stride, n_sel, wp, n, _f32(out, n, "out"), _stream(stream)), "qgemv_combine")


def qgemv_mapped_rows(w: Matrix, row_start: int, row_end: int, x, y, block_rows: int = 0,
                      stream=None) -> None:
    """As qgemv_rows, with ``w.data`` a pinned host tensor read in place over the host link."""
    m = w.c()
    n = max(row_end - row_start, 0)
    _check(lib().qgemv_mapped_rows(ctypes.byref(m), row_start, row_end, _f32(x, w.k, "x"), _f32(y, n, "y"),
                                   block_rows, _stream(stream)), "qgemv_mapped_rows")


def qgemv_mapped_windows(windows: Sequence[Window], block_rows: int = 0, stream=None, fmt=None, k=None) -> None:
    """As qgemv_windows, with every window's matrix in pinned host memory."""
    arr, n, f, kk = _windows(windows)
    f = fmt if f is None else f
    kk = k if kk is None else kk
    _check(lib().qgemv_mapped_windows(int(f or Q8_0), int(kk or 32), arr, n, block_rows, _stream(stream)),
           "qgemv_mapped_windows")


def qgemv_silu_mul(g, u, h, stream=None) -> None:
    n = h.numel()
    _check(lib().qgemv_silu_mul(_f32(g, n, "g"), _f32(u, n, "u"), _f32(h, n, "h"), n, _stream(stream)),
           "qgemv_silu_mul")


def qgemv_rms_carry(v, out, eps: float = 1e-6, gelu: bool = False, stream=None) -> None:
    n = v.numel()
    _check(lib().qgemv_rms_carry(_f32(v, n, "v"), _f32(out, n, "out"), n, float(eps), int(bool(gelu)),
                                 _stream(stream)), "qgemv_rms_carry")


def qgemv_read_ceiling(data, sink, stream=None) -> None:
    """One plain streaming read of the device tensor ``data`` (its whole
    storage; a multiple of 16 bytes); the xor of what was read is xor-ed into
    the uint32/int32 device tensor ``sink``."""
    n = data.numel() * data.element_size()
    if not data.is_cuda or not sink.is_cuda or sink.element_size() != 4:
        raise ValueError("data and sink must be device tensors, sink 32-bit")
    _check(lib().qgemv_read_ceiling(_ptr(data), n, _ptr(sink), _stream(stream)), "qgemv_read_ceiling")


def qgemv_dequant_rows(w: Matrix, row_start: int, row_end: int, out, stream=None) -> None:
    m = w.c()
    n = max(row_end - row_start, 0) * w.k
    _check(lib().qgemv_dequant_rows(ctypes.byref(m), row_start, row_end, _f32(out, n, "out"),
                                    _stream(stream)), "qgemv_dequant_rows")


class Streamer:
    """Owner of a qg_streamer: lookahead + 1 device slots of slot_bytes each."""

    def __init__(self, slot_bytes: int, lookahead: int):
        h = _vp()
        _check(lib().qgemv_stream_create(int(slot_bytes), int(lookahead), ctypes.byref(h)),
               "qgemv_stream_create")
        self._h = h
        self.slot_bytes = int(slot_bytes)
        self.lookahead = int(lookahead)

    @property
    def ring_bytes(self) -> int:
        return int(lib().qgemv_stream_ring_bytes(self._h))

    def rows(self, w: Matrix, row_start: int, row_end: int, x, y, block_rows: int = 0, stream=None) -> None:
        m = w.c()
        n = max(row_end - row_start, 0)
        _check(lib().qgemv_stream_rows(self._h, ctypes.byref(m), row_start, row_end, block_rows,
                                       _f32(x, w.k, "x"), _f32(y, n, "y"), _stream(stream)),
               "qgemv_stream_rows")

    def windows(self, windows: Sequence[Window], block_rows: int = 0, stream=None) -> None:
        arr, n, f, k = _windows(windows)
        _check(lib().qgemv_stream_windows(self._h, int(f or Q8_0), int(k or 32), arr, n, block_rows,
                                          _stream(stream)), "qgemv_stream_windows")

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            h, self._h = self._h, None
            _check(lib().qgemv_stream_destroy(h), "qgemv_stream_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


PLAN_GEMV, PLAN_SILU_MUL, PLAN_COMBINE = 1, 2, 3


@dataclass
class PlanGemv:
    """A streamed GEMV step of a plan: its windows (same fmt and k; data in
    pinned host memory) walked in blocks of block_rows."""
    windows: Sequence[Window]
    block_rows: int = 0


@dataclass
class PlanSiluMul:
    """h = silu(g) * u between the steps of a plan."""
    g: object
    u: object
    h: object


@dataclass
class PlanCombine:
    """out = sum_s w[s] y[s] (as qgemv_combine) between the steps of a plan."""
    y: object
    y_stride: int
    n_sel: int
    w: object
    n: int
    out: object


class StreamPlan:
    """Owner of a qg_stream_plan: a fixed walk of streamed GEMV steps and
    elementwise steps, replayed by run()."""

    def __init__(self, slot_bytes: int, lookahead: int, steps):
        wins, cs = [], []
        for st in steps:
            if isinstance(st, PlanGemv):
                first = len(wins)
                fmt, k = st.windows[0].mat.fmt, st.windows[0].mat.k
                wins.extend(st.windows)
                cs.append(qg_plan_step(PLAN_GEMV, int(fmt), int(k), first, len(st.windows), int(st.block_rows),
                                       None, None, None, 0, 0, 0, 0))
            elif isinstance(st, PlanSiluMul):
                n = st.h.numel()
                cs.append(qg_plan_step(PLAN_SILU_MUL, 0, 0, 0, 0, 0, _f32(st.g, n, "g"), _f32(st.u, n, "u"),
                                       _f32(st.h, n, "h"), n, 0, 0, 0))
            elif isinstance(st, PlanCombine):
                cs.append(qg_plan_step(PLAN_COMBINE, 0, 0, 0, 0, 0, _ptr(st.y), _ptr(st.w), _f32(st.out, st.n, "out"),
                                       int(st.n), int(st.y_stride), int(st.n_sel), 0))
            else:
                raise TypeError(f"not a plan step: {st!r}")
        sarr = (qg_plan_step * len(cs))(*cs)
        warr = (qg_window * max(len(wins), 1))(*[w.c() for w in wins])
        h = _vp()
        _check(lib().qgemv_stream_plan_create(int(slot_bytes), int(lookahead), sarr, len(cs), warr, len(wins),
                                              ctypes.byref(h)), "qgemv_stream_plan_create")
        self._h = h
        self._keep = list(steps)  # the tensors must outlive the plan

    @property
    def ring_bytes(self) -> int:
        return int(lib().qgemv_stream_plan_ring_bytes(self._h))

    def set_rows(self, w: int, row_start: int) -> None:
        _check(lib().qgemv_stream_plan_set_rows(self._h, int(w), int(row_start)), "qgemv_stream_plan_set_rows")

    def run(self, stream=None) -> None:
        _check(lib().qgemv_stream_plan_run(self._h, _stream(stream)), "qgemv_stream_plan_run")

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            h, self._h = self._h, None
            _check(lib().qgemv_stream_plan_destroy(h), "qgemv_stream_plan_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


NOALLOC_RING_BYTES = 32 << 20


def qgemv_stream_rows_noalloc(w: Matrix, row_start: int, row_end: int, x, y, block_rows: int = 0,
                              stream=None) -> None:
    """Streamed rows through the library's own two-slot ring (no allocation;
    blocks up to NOALLOC_RING_BYTES / 2 bytes; calls must not overlap on a GPU)."""
    m = w.c()
    n = max(row_end - row_start, 0)
    _check(lib().qgemv_stream_rows_noalloc(ctypes.byref(m), row_start, row_end, block_rows, _f32(x, w.k, "x"),
                                           _f32(y, n, "y"), _stream(stream)), "qgemv_stream_rows_noalloc")


def qgemv_stream_create(slot_bytes: int, lookahead: int) -> Streamer:
    return Streamer(slot_bytes, lookahead)


@dataclass
class ChainWindow:
    """Rows [row_start, row_end) of ``mat``: y = W[row_start:row_end] . op(x),
    op the step's input transform (``x2`` is the multiplier of IN_SILU_MUL)."""
    mat: Matrix
    row_start: int
    row_end: int
    x: object
    y: object
    x2: object = None


@dataclass
class ChainStep:
    """One step of a chain: its windows (same fmt and k) and input transform."""
    windows: Sequence[ChainWindow]
    in_op: int = IN_X
    eps: float = 1e-6


def _chain_tables(steps: Sequence[ChainStep]):
    wins, cs = [], []
    for st in steps:
        if not st.windows:
            raise ValueError("a chain step needs at least one window")
        k = st.windows[0].mat.k
        first = len(wins)
        for w in st.windows:
            if w.mat.k != k:
                raise ValueError("the windows of a chain step must share k")
            n = max(w.row_end - w.row_start, 0)
            x2 = _f32(w.x2, k, "x2") if w.x2 is not None else 0
            wins.append(qg_chain_window(_ptr(w.mat.data), int(w.mat.n_rows), int(w.row_start), int(w.row_end),
                                        _f32(w.x, k, "x"), x2, _f32(w.y, n, "y")))
        cs.append(qg_chain_step(int(k), first, len(st.windows), int(st.in_op), float(st.eps)))
    return (qg_chain_step * len(cs))(*cs), len(cs), (qg_chain_window * len(wins))(*wins), len(wins)


class Chain:
    """Owner of a qg_chain: the steps run in order by one launch per run()."""

    def __init__(self, fmt: int, steps: Sequence[ChainStep]):
        sarr, ns, warr, nw = _chain_tables(steps)
        h = _vp()
        _check(lib().qgemv_chain_create(int(fmt), sarr, ns, warr, nw, ctypes.byref(h)), "qgemv_chain_create")
        self._h = h
        self._keep = list(steps)  # the tensors must outlive the chain
        self.fmt = int(fmt)
        self.n_steps = ns

    @property
    def grid(self) -> int:
        return int(lib().qgemv_chain_grid(self._h))

    @property
    def handle(self) -> int:
        return int(self._h.value)

    def run(self, stream=None) -> None:
        _check(lib().qgemv_chain_run(self._h, _stream(stream)), "qgemv_chain_run")

    def check(self) -> None:
        _check(lib().qgemv_chain_check(self._h), "qgemv_chain_check")

    def set_spin_limit(self, polls: int) -> None:
        """Polls (>= 1) a barrier waits before it gives up (default 2^22)."""
        _check(lib().qgemv_chain_set_spin_limit(self._h, int(polls)), "qgemv_chain_set_spin_limit")

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            h, self._h = self._h, None
            _check(lib().qgemv_chain_destroy(h), "qgemv_chain_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def qgemv_chain_create(fmt: int, steps: Sequence[ChainStep]) -> Chain:
    return Chain(fmt, steps)


# --- prompts over MXFP4 weights (include/qgemv_mx.h) -------------------------------
#
# Activations are 2-D device tensors of float32, float16 or bfloat16 with unit
# column stride (any row stride), or MXFP4 blocks as a Matrix.  Every tensor of
# a call must lie on the current device.

# A small call's time is the host's: names of torch are looked up once, and a
# tensor's device is compared with the driver's current one without a
# torch.cuda call each (a token's sort, gather and weighted sum 18.7 us, not 24.3).
_kinds = _int32 = _float32 = _float64 = _device = _raw_stream = None


def _torch_names() -> None:
    global _kinds, _int32, _float32, _float64, _device, _raw_stream
    import torch
    _int32, _float32, _float64 = torch.int32, torch.float32, torch.float64
    _device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _kinds = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


def _here(t, name: str) -> int:
    """The tensor's address, checked to be on the current device."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a device tensor")
    if d != _device():
        raise ValueError(f"{name} is on cuda:{d}, the current device is cuda:{_device()}")
    return t.data_ptr()


def _here_stream(stream) -> int:
    """As _stream, after a tensor was found on the device."""
    return _raw_stream(_device()) if stream is None else _stream(stream)


def _rows(t, name: str) -> qg_tensor:
    """A qg_tensor of a 2-D float tensor, or of a Matrix of blocks."""
    if isinstance(t, Matrix):
        return qg_tensor(_blocks(t, name).data, int(t.fmt), 0, int(t.n_rows), int(t.k), int(t.k))
    if _kinds is None:
        _torch_names()
    kind = _kinds.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    n, cols = shape
    stride, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    # (the stride of a single row says nothing)
    return qg_tensor(_here(t, name), kind, 0, n, cols, stride if n > 1 else cols)


def _blocks(m: Matrix, name: str) -> qg_matrix:
    """A qg_matrix whose blocks are on the current device and all there."""
    if _kinds is None:
        _torch_names()
    data, n, k = m.data, int(m.n_rows), int(m.k)
    p = _here(data, name)
    if not data.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    n_bytes = data.nbytes
    if m.fmt == MXFP4 and k > 0 and k % 32 == 0 and n_bytes < n * (k // 32 * 17):
        raise ValueError(f"{name} holds {n_bytes} bytes, needs {n * (k // 32 * 17)}")
    return qg_matrix(p, int(m.fmt), 0, n, k, n_bytes)


def _array(t, n: int, name: str, dtype, type_name: str) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {type_name}")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} values, needs {n}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _here(t, name)


def _i32s(t, n: int, name: str) -> int:
    if _kinds is None:
        _torch_names()
    return _array(t, n, name, _int32, "int32")


def _weights(t, n: int, name: str) -> int:
    if _kinds is None:
        _torch_names()
    return _array(t, n, name, _float32, "float32")


def _n_sel(n) -> int:
    """A number of choices for a C int: past 32 bits, where ctypes would cut it, the largest, which is refused or
    makes every slot the first token's as the number itself would."""
    return max(min(int(n), 0x7fffffff), -1)


def _per_choice(t, pos, name: str) -> int:
    """The address of one float32 per (token, choice) of ``pos``: flat, or of rows of as many choices."""
    n_tok, n_sel = pos.shape
    if t.dim() > 1 and t.shape[-1] != n_sel and n_tok > 1 and n_sel > 1:
        raise ValueError(f"{name} must be (tokens, choices)")
    return _weights(t, n_tok * n_sel, name)


def qgemv_mx_quantize(x, q: Matrix, stream=None) -> None:
    """Quantises the rows of ``x`` into the MXFP4 blocks of ``q`` (n_rows x k of x's shape)."""
    _check(lib().qgemv_mx_quantize(ctypes.byref(_rows(x, "x")), ctypes.byref(_blocks(q, "q")), _here_stream(stream)),
           "qgemv_mx_quantize")


def qgemv_mx_dequantize(q: Matrix, row_start: int, row_end: int, out, stream=None) -> None:
    """The values of rows [row_start, row_end) of ``q``, rounded to out's type."""
    _check(lib().qgemv_mx_dequantize(ctypes.byref(_blocks(q, "q")), row_start, row_end,
                                     ctypes.byref(_rows(out, "out")), _here_stream(stream)), "qgemv_mx_dequantize")


def qgemv_rows_mx(w: Matrix, row_start: int, row_end: int, x, y, stream=None) -> None:
    """y[t] = W[row_start:row_end] . x[t] for any number of tokens; ``x`` a float
    tensor (tokens, k) or an MXFP4 Matrix, ``y`` (tokens, rows) of any float type."""
    _check(lib().qgemv_rows_mx(ctypes.byref(_blocks(w, "w")), row_start, row_end, ctypes.byref(_rows(x, "x")),
                               ctypes.byref(_rows(y, "y")), _here_stream(stream)), "qgemv_rows_mx")


def qgemv_rows_mx_swiglu(gate: Matrix, up: Matrix, row_start: int, row_end: int, x, h, stream=None) -> None:
    """h = silu(gate[rows] . x) * (up[rows] . x), as qgemv_rows_mx."""
    _check(lib().qgemv_rows_mx_swiglu(ctypes.byref(_blocks(gate, "gate")), ctypes.byref(_blocks(up, "up")), row_start,
                                      row_end, ctypes.byref(_rows(x, "x")), ctypes.byref(_rows(h, "h")),
                                      _here_stream(stream)), "qgemv_rows_mx_swiglu")


def qgemv_expert_sort(ids, n_expert: int, offsets, slots, pos, stream=None) -> None:
    """Stable sort of the slots of ``ids`` (tokens, choices; int32) by expert:
    ``offsets`` (n_expert + 1), ``slots`` and ``pos`` (one per slot), int32."""
    if ids.dim() != 2:
        raise ValueError("ids must be (tokens, choices)")
    n_tok, n_sel = ids.shape
    n = n_tok * n_sel
    _check(lib().qgemv_expert_sort(_i32s(ids, n, "ids"), n_tok, _n_sel(n_sel), int(n_expert),
                                   _i32s(offsets, max(int(n_expert), 0) + 1, "offsets"), _i32s(slots, n, "slots"),
                                   _i32s(pos, n, "pos"), _here_stream(stream)), "qgemv_expert_sort")


def _expert_args(x, n_expert: int, offsets, y, slots, n_sel):
    yt = _rows(y, "y")
    if slots is None:
        sp, n_sel = None, 1
    elif n_sel is None:
        raise ValueError("slots need n_sel, the choices of a token that the sort was given")
    else:
        sp = _i32s(slots, yt.n_rows, "slots")
    return (ctypes.byref(_rows(x, "x")), _i32s(offsets, max(int(n_expert), 0) + 1, "offsets"), sp, _n_sel(n_sel),
            ctypes.byref(yt))


def qgemv_expert_mx(w: Matrix, n_expert: int, x, offsets, y, slots=None, n_sel=None, stream=None) -> None:
    """y[p] = W_e . x[src] for the sorted places p of every expert e; src =
    slots[p] // n_sel (required with ``slots``), or p without ``slots``.  Rows
    of y behind the last place stay."""
    xt, op, sp, ns, yt = _expert_args(x, n_expert, offsets, y, slots, n_sel)
    _check(lib().qgemv_expert_mx(ctypes.byref(_blocks(w, "w")), int(n_expert), xt, op, sp, ns, yt,
                                 _here_stream(stream)), "qgemv_expert_mx")


def qgemv_expert_mx_swiglu(gate: Matrix, up: Matrix, n_expert: int, x, offsets, h, slots=None, n_sel=None,
                           stream=None) -> None:
    """h[p] = silu(gate_e . x[src]) * (up_e . x[src]), as qgemv_expert_mx."""
    xt, op, sp, ns, ht = _expert_args(x, n_expert, offsets, h, slots, n_sel)
    _check(lib().qgemv_expert_mx_swiglu(ctypes.byref(_blocks(gate, "gate")), ctypes.byref(_blocks(up, "up")),
                                        int(n_expert), xt, op, sp, ns, ht, _here_stream(stream)),
           "qgemv_expert_mx_swiglu")


def qgemv_expert_gather(x, slots, n_sel: int, out, stream=None) -> None:
    """out[p] = x[slots[p] // n_sel]; rows with a negative slot stay."""
    ot = _rows(out, "out")
    _check(lib().qgemv_expert_gather(ctypes.byref(_rows(x, "x")), _i32s(slots, ot.n_rows, "slots"), _n_sel(n_sel),
                                     ctypes.byref(ot), _here_stream(stream)), "qgemv_expert_gather")


def qgemv_expert_combine(y, pos, out, w=None, stream=None) -> None:
    """out[t] = sum_s w[t, s] y[pos[t, s]]; without ``w`` the weights are 1 (the
    gather's gradient).  ``pos`` and ``w`` are (tokens, choices)."""
    if pos.dim() != 2 or pos.shape[0] != out.shape[0]:
        raise ValueError("pos must be (tokens, choices) with out's tokens")
    _check(lib().qgemv_expert_combine(ctypes.byref(_rows(y, "y")), _i32s(pos, pos.numel(), "pos"),
                                      _per_choice(w, pos, "w") if w is not None else None, _n_sel(pos.shape[1]),
                                      ctypes.byref(_rows(out, "out")), _here_stream(stream)), "qgemv_expert_combine")


def qgemv_expert_combine_grad(dout, y, pos, w, dy, dw, stream=None) -> None:
    """The gradient of qgemv_expert_combine: dy[pos[t, s]] = w[t, s] dout[t],
    dw[t, s] = <dout[t], y[pos[t, s]]> (float32)."""
    if pos.dim() != 2 or pos.shape[0] != dout.shape[0]:
        raise ValueError("pos must be (tokens, choices) with dout's tokens")
    _check(lib().qgemv_expert_combine_grad(ctypes.byref(_rows(dout, "dout")), ctypes.byref(_rows(y, "y")),
                                           _i32s(pos, pos.numel(), "pos"), _per_choice(w, pos, "w"), _n_sel(pos.shape[1]),
                                           ctypes.byref(_rows(dy, "dy")), _per_choice(dw, pos, "dw"),
                                           _here_stream(stream)),
           "qgemv_expert_combine_grad")


# --- a paged cache of keys and values (include/qgemv_kv.h) ---------------------------
#
# Activations are 3-D device tensors (tokens, heads, head_dim) of float32, float16
# or bfloat16 with unit last stride: slices of a QKV product's rows as they are.
# Every tensor of a call must lie on the current device.

@dataclass
class Rope:
    """Rotary positions: ``freqs`` (device, float64; n_rot / 2 radians a position), pairs (i, i + n_rot / 2) or,
    ``interleaved``, (2 i, 2 i + 1), turned values times ``mscale``."""
    freqs: object
    interleaved: bool = False
    mscale: float = 1.0


@dataclass
class KvCache:
    """Keys and values: device tensors (layers, pages, heads, page_size, head_dim), float16 or bfloat16, of the same
    strides (any order of the axes but the last in memory)."""
    k: object
    v: object


@dataclass
class KvSeqs:
    """Sequences of a call, int32 device tensors: ``starts`` (n_seq + 1) the first rows of their new tokens, ``lens``
    (n_seq) their positions with the new ones, ``tables`` (n_seq, max_pages) their pages."""
    starts: object
    lens: object
    tables: object


@dataclass
class KvPool:
    """Who holds which page, int32 device tensors that the calls keep up to date: ``tables`` (n_seq, max_pages; -1
    behind a sequence's length), ``lens`` (n_seq), ``refs`` (n_pages), ``used`` (a bit a page); ``work`` of
    qgemv_kv_pool_bytes."""
    tables: object
    lens: object
    refs: object
    used: object
    page_size: int
    work: object


# (packed as the header's structs: a ctypes.Structure takes several times as long to make; a decoded token's append
# 15.4 -> 10.6 us a call)
_HEADS, _ROPE, _CACHE = struct.Struct("Piiqiiqq"), struct.Struct("Piid"), struct.Struct("PPiiiiiiqqqqq")
_SEQS, _POOL = struct.Struct("PPPiiq"), struct.Struct("PPPPiiqqPq")


def _on(t, dev: int, name: str) -> int:
    """The tensor's address, checked to be on the device that is current."""
    if t.get_device() != dev:
        _here(t, name)
    return t.data_ptr()


def _current() -> int:
    if _kinds is None:
        _torch_names()
    return _device()


def _heads(t, dev: int, name: str) -> bytes:
    kind = _kinds.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be (tokens, heads, head_dim)")
    tok, head, unit = t.stride()
    if unit != 1 and shape[2] > 1:
        raise ValueError(f"the heads of {name} must be contiguous")
    return _HEADS.pack(_on(t, dev, name), kind, 0, *shape, tok, head)


def _ints(t, n: int, dev: int, name: str) -> int:
    if t.dtype is not _int32:
        raise TypeError(f"{name} must be int32")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} values, needs {n}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _on(t, dev, name)


def _c32(n) -> int:
    """A number for a C int: past 32 bits, where it would be cut, the largest, which is refused (as a window it is the
    widest)."""
    return max(min(int(n), 0x7fffffff), -0x80000000)


def _rope(r: Rope, dev: int) -> bytes:
    f = r.freqs
    if f.dtype is not _float64 or f.dim() != 1 or not f.is_contiguous():
        raise TypeError("freqs must be a contiguous float64 vector")
    return _ROPE.pack(_on(f, dev, "freqs"), 2 * f.numel(), bool(r.interleaved), r.mscale)


def _cache(c: KvCache, dev: int) -> bytes:
    k, v = c.k, c.v
    kind = _kinds.get(k.dtype)
    if kind is None:
        raise TypeError(f"the cache must be float16 or bfloat16, not {k.dtype}")
    shape, strides = k.shape, k.stride()
    if len(shape) != 5:
        raise ValueError("the cache must be (layers, pages, heads, page_size, head_dim)")
    if v.dtype is not k.dtype or v.shape != shape or v.stride() != strides:
        raise ValueError("k and v of the cache must have the same type, sizes and strides")
    layer, page, head, slot, unit = strides
    if unit != 1:
        raise ValueError("the heads of the cache must be contiguous")
    layers, pages, heads, size, dim = shape
    return _CACHE.pack(_on(k, dev, "k"), _on(v, dev, "v"), kind, size, layers, heads, dim, 0, pages, layer, page, head,
                       slot)


def _seqs(s: KvSeqs, dev: int) -> bytes:
    n, pages = s.tables.shape
    return _SEQS.pack(_ints(s.starts, n + 1, dev, "starts"), _ints(s.lens, n, dev, "lens"),
                      _ints(s.tables, n * pages, dev, "tables"), n, 0, pages)


def _pool(p: KvPool, dev: int) -> bytes:
    n, pages = p.tables.shape
    n_pages = p.refs.numel()
    return _POOL.pack(_ints(p.tables, n * pages, dev, "tables"), _ints(p.lens, n, dev, "lens"),
                      _ints(p.refs, n_pages, dev, "refs"), _ints(p.used, (n_pages + 31) // 32, dev, "used"), n,
                      _c32(p.page_size), pages, n_pages, *_work(p.work, dev))


def _work(t, dev: int):
    if t is None:
        return 0, 0
    if not t.is_contiguous():
        raise ValueError("work must be contiguous")
    return _on(t, dev, "work"), t.nbytes


def _floats(t, n: int, dev: int, name: str) -> int:
    if t.dtype is not _float32:
        raise TypeError(f"{name} must be float32")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} values, needs {n}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _on(t, dev, name)


def qgemv_rope_freqs(n_rot: int, base: float = 10000.0, scaling: int = ROPE_NONE, factor: float = 1.0,
                     trained: float = 4096.0, fast: float = 32.0, slow: float = 1.0):
    """(frequencies as a list of n_rot / 2 floats, mscale) of rotary positions of ``base``, stretched by ``factor``."""
    out, m = (_f64 * max(int(n_rot) // 2, 1))(), _f64()
    _check(lib().qgemv_rope_freqs(_c32(n_rot), base, int(scaling), factor, trained, fast, slow, out, ctypes.byref(m)),
           "qgemv_rope_freqs")
    return list(out), m.value


def qgemv_rope(x, pos, rope: Rope, y, inverse: bool = False, stream=None) -> None:
    """y[t] = x[t] turned by its position ``pos[t]`` (int32), or ``inverse`` by -pos[t], the turn's gradient; ``y``
    may be ``x``."""
    dev = _current()
    _check(lib().qgemv_rope(_heads(x, dev, "x"), _ints(pos, x.shape[0], dev, "pos"), _rope(rope, dev),
                            _heads(y, dev, "y"), bool(inverse), _here_stream(stream)), "qgemv_rope")


def qgemv_kv_append(k, v, seqs: KvSeqs, cache: KvCache, layer: int, rope: Rope = None, pos=None, q=None, q_out=None,
                    stream=None) -> None:
    """The new tokens' keys, turned by ``rope``, and values into ``layer`` of the cache, and ``q`` turned into
    ``q_out``; by their positions in the sequence, or by ``pos`` (int32, one a row)."""
    dev = _current()
    _check(lib().qgemv_kv_append(_heads(k, dev, "k"), _heads(v, dev, "v"), _seqs(seqs, dev), _cache(cache, dev),
                                 _c32(layer), _rope(rope, dev) if rope is not None else None,
                                 _ints(pos, k.shape[0], dev, "pos") if pos is not None else None,
                                 _heads(q, dev, "q") if q is not None else None,
                                 _heads(q_out, dev, "q_out") if q_out is not None else None, _here_stream(stream)),
           "qgemv_kv_append")


def qgemv_kv_attend_bytes(q, seqs: KvSeqs, cache: KvCache) -> int:
    """Bytes of ``work`` for a qgemv_kv_attend of these sizes (a smaller call may need more)."""
    dev = _current()
    n = lib().qgemv_kv_attend_bytes(_heads(q, dev, "q"), _seqs(seqs, dev), _cache(cache, dev))
    if n < 0:
        _check(n, "qgemv_kv_attend_bytes")
    return n


def qgemv_kv_attend(q, seqs: KvSeqs, cache: KvCache, layer: int, out, scale: float, causal: bool = True,
                    window: int = 0, sinks=None, lse=None, work=None, stream=None) -> None:
    """out = softmax(scale q k^T) v of the new tokens over their sequences' positions in ``layer``; ``sinks`` (float32,
    one a q head), ``lse`` (float32, tokens x q heads) and ``work`` (qgemv_kv_attend_bytes) as the header has them."""
    dev = _current()
    n, heads, _ = q.shape
    _check(lib().qgemv_kv_attend(_heads(q, dev, "q"), _seqs(seqs, dev), _cache(cache, dev), _c32(layer),
                                 _heads(out, dev, "out"), scale, bool(causal), _c32(window),
                                 _floats(sinks, heads, dev, "sinks") if sinks is not None else None,
                                 _floats(lse, n * heads, dev, "lse") if lse is not None else None, *_work(work, dev),
                                 _here_stream(stream)), "qgemv_kv_attend")


def qgemv_kv_pool_bytes(n_seq: int, max_pages: int, n_pages: int) -> int:
    """Bytes of a pool's ``work``."""
    n = lib().qgemv_kv_pool_bytes(n_seq, max_pages, n_pages)
    if n < 0:
        _check(n, "qgemv_kv_pool_bytes")
    return n


def qgemv_kv_resize(pool: KvPool, cache: KvCache, lens, stream=None) -> None:
    """Cuts and grows the sequences to ``lens`` (int32; negative: as it is), copying shared pages they grow into;
    ``pool.lens`` tells which found room."""
    dev = _current()
    _check(lib().qgemv_kv_resize(_pool(pool, dev), _cache(cache, dev), _ints(lens, pool.tables.shape[0], dev, "lens"),
                                 _here_stream(stream)), "qgemv_kv_resize")


def qgemv_kv_fork(pool: KvPool, parents, stream=None) -> None:
    """All at once every sequence s becomes what ``parents[s]`` (int32) was, sharing its pages; -1 lets s go."""
    dev = _current()
    _check(lib().qgemv_kv_fork(_pool(pool, dev), _ints(parents, pool.tables.shape[0], dev, "parents"),
                               _here_stream(stream)), "qgemv_kv_fork")


def qgemv_kv_compact(pool: KvPool, cache: KvCache, stream=None) -> None:
    """Moves the pages in use to the lowest numbers."""
    dev = _current()
    _check(lib().qgemv_kv_compact(_pool(pool, dev), _cache(cache, dev), _here_stream(stream)), "qgemv_kv_compact")


def qgemv_kv_copy(cache: KvCache, src, dst, stream=None) -> None:
    """Page src[i] to page dst[i] (int32) in every layer."""
    dev = _current()
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src and dst must be of the same length")
    _check(lib().qgemv_kv_copy(_cache(cache, dev), _ints(src, n, dev, "src"), _ints(dst, n, dev, "dst"), n,
                               _here_stream(stream)), "qgemv_kv_copy")


def qgemv_version() -> str:
    return lib().qgemv_version().decode()
