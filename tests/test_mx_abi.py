"""include/qgemv_mx.h on the host (no GPU): every entry point is exported, bad
arguments are refused with the documented status before any HIP call, the
binding refuses what it cannot pass on, and the tests' plain forms hold."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import mxref
import quantized_gemv_gguf_amd as q
from quantized_gemv_gguf_amd import qg_matrix, qg_tensor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qgemv_mx.h")
E_NULL, E_FMT, E_SHAPE, E_RANGE, E_SIZE, E_ARG = -1, -2, -3, -4, -5, -6
FAKE = 0x1000  # a non-NULL address; never dereferenced by a call that is refused


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qgemv_\w+)\s*\(", text)))
    assert len(names) == 10, names
    out = subprocess.run(["nm", "-D", "--defined-only", q.LIB_PATH], capture_output=True, text=True).stdout
    exported = set(re.findall(r"\sT\s(\w+)$", out, flags=re.M))
    assert not [n for n in names if n not in exported]
    for n in names:
        assert hasattr(q.lib(), n) and hasattr(q, n)


def test_header_compiles_as_c_and_matches_the_binding():
    src = ('#include "qgemv_mx.h"\nint main(void){qg_tensor t; (void)t;'
           ' return sizeof(qg_tensor) == 40 && QG_F32 == %d && QG_F16 == %d && QG_BF16 == %d'
           ' && QG_MAX_EXPERTS == %d ? 0 : 1;}\n' % (q.F32, q.F16, q.BF16, q.MAX_EXPERTS))
    exe = "/tmp/qgemv_mx_header_%d" % os.getpid()
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", f"-I{os.path.dirname(HEADER)}", "-x", "c", "-",
                        "-o", exe], input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    try:
        assert subprocess.run([exe]).returncode == 0
    finally:
        os.remove(exe)
    assert ctypes.sizeof(qg_tensor) == 40


def mat(rows=8, k=64, fmt=3, data=FAKE, nbytes=None, reserved=0):
    return ctypes.byref(qg_matrix(data, fmt, reserved, rows, k, rows * (k // 32) * 17 if nbytes is None else nbytes))


def ten(rows=4, cols=64, kind=32, stride=None, data=FAKE, reserved=0):
    return ctypes.byref(qg_tensor(data, kind, reserved, rows, cols, cols if stride is None else stride))


# a tensor argument that every call refuses, and the status (as the input of a product with k = 64)
BAD_X = [(None, E_NULL), (ten(kind=0), E_FMT), (ten(kind=1), E_FMT), (ten(rows=-1), E_SHAPE), (ten(cols=-64), E_SHAPE),
         (ten(rows=1 << 31), E_SHAPE), (ten(cols=32), E_SHAPE), (ten(reserved=1), E_ARG), (ten(stride=-1), E_ARG),
         (ten(stride=(1 << 40) + 1), E_ARG), (ten(data=0), E_NULL), (ten(data=FAKE + 2), E_ARG),
         (ten(kind=33, data=FAKE + 1), E_ARG), (ten(kind=3, data=FAKE + 8), E_ARG), (ten(kind=3, stride=96), E_ARG),
         (ten(kind=3, cols=48), E_SHAPE)]
BAD_Y = [(None, E_NULL), (ten(cols=8, kind=3), E_FMT), (ten(cols=8, kind=31), E_FMT), (ten(cols=7), E_SHAPE),
         (ten(cols=8, rows=5), E_SHAPE), (ten(cols=8, stride=7), E_ARG), (ten(cols=8, data=0), E_NULL),
         (ten(cols=8, reserved=9), E_ARG), (ten(cols=8, kind=34, data=FAKE + 1), E_ARG)]
BAD_W = [(None, E_NULL), (mat(fmt=1, nbytes=8 * 2 * 34), E_FMT), (mat(fmt=0), E_FMT), (mat(k=0, nbytes=0), E_SHAPE),
         (mat(k=48, nbytes=0), E_SHAPE), (mat(k=49152 + 32), E_SHAPE), (mat(rows=-1), E_SHAPE),
         (mat(rows=1 << 31), E_SHAPE), (mat(reserved=2), E_ARG), (mat(nbytes=8 * 2 * 17 - 1), E_SIZE),
         (mat(data=0), E_NULL), (mat(data=FAKE + 4), E_ARG)]


def test_products_refuse():
    L = q.lib()
    for w, status in BAD_W:
        assert L.qgemv_rows_mx(w, 0, 8, ten(), ten(cols=8), None) == status
        assert L.qgemv_rows_mx_swiglu(w, mat(), 0, 8, ten(), ten(cols=8), None) == status
        assert L.qgemv_rows_mx_swiglu(mat(), w, 0, 8, ten(), ten(cols=8), None) == status
        assert L.qgemv_expert_mx(w, 2, ten(), FAKE, FAKE, 2, ten(cols=4), None) == status
        assert L.qgemv_expert_mx_swiglu(mat(), w, 2, ten(), FAKE, FAKE, 2, ten(cols=4), None) == status
    for x, status in BAD_X:
        assert L.qgemv_rows_mx(mat(), 0, 8, x, ten(cols=8), None) == status
        assert L.qgemv_rows_mx_swiglu(mat(), mat(), 0, 8, x, ten(cols=8), None) == status
        assert L.qgemv_expert_mx(mat(16), 2, x, FAKE, FAKE, 2, ten(cols=8), None) == status
    for y, status in BAD_Y:
        assert L.qgemv_rows_mx(mat(), 0, 8, ten(), y, None) == status
        assert L.qgemv_rows_mx_swiglu(mat(), mat(), 0, 8, ten(), y, None) == status
    for r0, r1 in [(-1, 8), (5, 4), (0, 9)]:
        assert L.qgemv_rows_mx(mat(), r0, r1, ten(), ten(cols=8), None) == E_RANGE
    assert L.qgemv_rows_mx_swiglu(mat(), mat(9), 0, 8, ten(), ten(cols=8), None) == E_SHAPE
    assert L.qgemv_rows_mx_swiglu(mat(), mat(k=96), 0, 8, ten(), ten(cols=8), None) == E_SHAPE
    # nothing to do: no HIP call, no data
    assert L.qgemv_rows_mx(mat(), 3, 3, ten(), ten(cols=0, data=0), None) == 0
    assert L.qgemv_rows_mx(mat(), 0, 8, ten(rows=0, data=0), ten(rows=0, cols=8, data=0), None) == 0


def test_largest_sizes():
    """Past 2^31 - 2^16 rows or columns, where a tile's last index would leave 32 bits, and past 2^30 choices."""
    L = q.lib()
    for rows in (2 ** 31 - 2 ** 16 + 1, 2 ** 31 - 1):
        assert L.qgemv_rows_mx(mat(), 0, 8, ten(rows=rows), ten(rows=rows, cols=8), None) == E_SHAPE
        assert L.qgemv_rows_mx(mat(rows), 0, rows, ten(), ten(cols=rows), None) == E_SHAPE
        assert L.qgemv_expert_mx(mat(16), 2, ten(), FAKE, FAKE, 2, ten(rows=rows, cols=8), None) == E_SHAPE
        assert L.qgemv_mx_quantize(ten(rows=rows), mat(rows), None) == E_SHAPE
        assert L.qgemv_mx_dequantize(mat(rows), 0, rows, ten(rows=rows), None) == E_SHAPE
        assert L.qgemv_expert_gather(ten(), FAKE, 2, ten(rows=rows), None) == E_SHAPE
        assert L.qgemv_expert_combine(ten(cols=rows), FAKE, FAKE, 2, ten(cols=rows), None) == E_SHAPE
    assert L.qgemv_expert_combine(ten(), FAKE, FAKE, 2 ** 30 + 1, ten(rows=1), None) == E_SHAPE
    # (the largest that are taken, without work)
    most = 2 ** 31 - 2 ** 16
    assert L.qgemv_rows_mx(mat(most), 5, 5, ten(), ten(cols=0, data=0), None) == 0
    assert L.qgemv_expert_combine(ten(cols=0), FAKE, FAKE, 2 ** 30, ten(cols=0), None) == 0


def test_expert_products_refuse():
    L = q.lib()

    def call(w=None, e=2, x=None, offsets=FAKE, slots=FAKE, sel=2, y=None):
        return L.qgemv_expert_mx(w or mat(16), e, x or ten(), offsets, slots, sel, y or ten(rows=6, cols=8), None)

    assert call(e=0) == E_SHAPE and call(e=-1) == E_SHAPE and call(e=1025) == E_SHAPE
    assert call(e=3) == E_SHAPE                                   # 16 rows are not three experts'
    assert call(y=ten(rows=6, cols=16)) == E_SHAPE
    assert call(x=ten(cols=96)) == E_SHAPE
    assert call(sel=0) == E_ARG and call(sel=-2) == E_ARG
    assert call(offsets=None) == E_NULL
    assert call(slots=None) == E_SHAPE                            # 4 rows of x for 6 places
    assert call(slots=None, x=ten(rows=6), offsets=None) == E_NULL
    assert call(y=ten(rows=0, cols=8, data=0), offsets=None, slots=None) == 0
    assert call(w=mat(0, data=0), y=ten(rows=6, cols=0, data=0)) == 0


def test_quantisation_refuses():
    L = q.lib()
    for x, status in BAD_X[:-3]:
        assert L.qgemv_mx_quantize(x, mat(4), None) == status
    assert L.qgemv_mx_quantize(ten(kind=3), mat(4), None) == E_FMT
    assert L.qgemv_mx_quantize(ten(rows=5), mat(4), None) == E_SHAPE
    for w, status in BAD_W:
        assert L.qgemv_mx_quantize(ten(rows=8), w, None) == status
        assert L.qgemv_mx_dequantize(w, 0, 8, ten(rows=8), None) == status
    assert L.qgemv_mx_dequantize(mat(), 0, 9, ten(rows=9), None) == E_RANGE
    assert L.qgemv_mx_dequantize(mat(), 0, 8, ten(rows=7), None) == E_SHAPE
    assert L.qgemv_mx_dequantize(mat(), 0, 8, ten(rows=8, stride=63), None) == E_ARG
    assert L.qgemv_mx_dequantize(mat(), 0, 8, ten(rows=8, kind=3), None) == E_FMT
    assert L.qgemv_mx_quantize(ten(rows=0, data=0), mat(0, data=0), None) == 0
    assert L.qgemv_mx_dequantize(mat(), 4, 4, ten(rows=0, data=0), None) == 0


def test_routing_refuses():
    L = q.lib()
    sort = L.qgemv_expert_sort
    assert sort(FAKE, -1, 2, 4, FAKE, FAKE, FAKE, None) == E_ARG
    assert sort(FAKE, 4, 0, 4, FAKE, FAKE, FAKE, None) == E_ARG
    assert sort(FAKE, 4, 2, 0, FAKE, FAKE, FAKE, None) == E_SHAPE
    assert sort(FAKE, 4, 2, 1025, FAKE, FAKE, FAKE, None) == E_SHAPE
    assert sort(FAKE, (1 << 29) + 1, 2, 4, FAKE, FAKE, FAKE, None) == E_SHAPE
    for i in (0, 4, 5, 6):
        args = [FAKE, 4, 2, 4, FAKE, FAKE, FAKE, None]
        args[i] = None
        assert sort(*args) == E_NULL
    gather = L.qgemv_expert_gather
    assert gather(ten(), FAKE, 2, ten(kind=34), None) == E_FMT
    assert gather(ten(), FAKE, 2, ten(cols=65), None) == E_SHAPE
    assert gather(ten(), FAKE, 0, ten(), None) == E_ARG
    assert gather(ten(), None, 2, ten(), None) == E_NULL
    assert gather(ten(kind=3), FAKE, 2, ten(kind=3), None) == E_FMT
    assert gather(ten(), None, 2, ten(rows=0, data=0), None) == 0
    combine = L.qgemv_expert_combine
    assert combine(ten(), FAKE, FAKE, 2, ten(cols=65), None) == E_SHAPE
    assert combine(ten(), FAKE, FAKE, -1, ten(), None) == E_ARG
    assert combine(ten(), None, FAKE, 2, ten(), None) == E_NULL
    assert combine(ten(), FAKE, FAKE, 2, ten(stride=63), None) == E_ARG
    assert combine(ten(), None, None, 2, ten(rows=0, data=0), None) == 0
    grad = L.qgemv_expert_combine_grad
    other = dict(data=2 * FAKE)
    assert grad(ten(), ten(rows=8), FAKE, FAKE, 2, ten(rows=8, kind=34), FAKE, None) == E_FMT
    assert grad(ten(), ten(rows=8), FAKE, FAKE, 2, ten(rows=7), FAKE, None) == E_SHAPE
    assert grad(ten(), ten(rows=8), FAKE, FAKE, 0, ten(rows=8, **other), FAKE, None) == E_ARG
    assert grad(ten(), ten(rows=8), FAKE, FAKE, 2, ten(rows=8), FAKE, None) == E_ARG  # dy on y
    for i in (2, 3, 6):
        args = [ten(), ten(rows=8), FAKE, FAKE, 2, ten(rows=8, **other), FAKE, None]
        args[i] = None
        assert grad(*args) == E_NULL


def test_binding_refuses():
    import torch
    x = torch.zeros(2, 64)
    w = q.Matrix(torch.zeros(8 * 34, dtype=torch.uint8), q.MXFP4, 8, 64)
    with pytest.raises(ValueError, match="device tensor"):
        q.qgemv_rows_mx(w, 0, 8, x, torch.zeros(2, 8), stream=0)
    with pytest.raises(ValueError, match="device tensor"):
        q.qgemv_mx_quantize(x, w, stream=0)
    with pytest.raises(TypeError, match="float"):
        q.qgemv_expert_gather(x.double(), torch.zeros(2, dtype=torch.int32), 1, x.double(), stream=0)
    with pytest.raises(ValueError, match="2-D"):
        q.qgemv_expert_gather(x[0], torch.zeros(2, dtype=torch.int32), 1, x[0], stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        q.qgemv_expert_gather(x.t(), torch.zeros(2, dtype=torch.int32), 1, x.t(), stream=0)
    with pytest.raises(TypeError, match="int32"):
        q.qgemv_expert_sort(torch.zeros(2, 2, dtype=torch.int64), 2, x, x, x, stream=0)
    with pytest.raises(ValueError, match="ids"):
        q.qgemv_expert_sort(torch.zeros(4, dtype=torch.int32), 2, x, x, x, stream=0)


def test_plain_quantisation_against_its_definition():
    """The plain form of the tests: nearest grid value at the block's scale, ties to even codes, a constant
    block of each code, zeros, infinities and subnormals."""
    grid = mxref.GRID
    x = np.concatenate([grid, -grid, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], np.zeros(8)])[None]
    v = mxref.values(mxref.quantize(x), 32)[0]
    assert np.array_equal(v[:16], x[0, :16])
    assert np.array_equal(v[16:24], [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0])
    assert mxref.quantize(np.zeros((1, 32)))[0, 0] == 0
    b = mxref.quantize(np.full((1, 32), 2.0 ** -140))
    assert b[0, 0] == 0 and not b[0, 1:].any()
    for bad in (np.inf, -np.inf, np.nan):
        y = np.ones((1, 64))
        y[0, 40] = bad
        b = mxref.quantize(y)
        assert b[0, 0] == 125 and b[0, 17] == 255
        assert np.isnan(mxref.values(b, 64)[0, 32:]).all() and (mxref.values(b, 64)[0, :32] == 1).all()


def test_plain_sort():
    offsets, slots, pos = mxref.sort(np.array([[2, 0], [-1, 2], [5, 0]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert slots.tolist() == [1, 5, 0, 3, -1, -1]
    assert pos.tolist() == [[2, 0], [-1, 3], [-1, 1]]
