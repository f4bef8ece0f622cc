"""What the bits of an MXFP4 product (include/qgemv_mx.h) depend on: not on where
a window of rows begins, nor on how places are shared among the experts; and
windows of other sizes agree within the bounds of their sums."""
from __future__ import annotations

import numpy as np
import pytest

import mxref
import quantized_gemv_gguf_amd as q
from test_gpu_mx import activations, blocks, dput, host, nan_buffer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("tok,n,k", [(1, 300, 416), (16, 1100, 2880), (40, 300, 416), (700, 1030, 224)])
def test_windows(dev, kind, pair, tok, n, k):
    rng = np.random.default_rng(tok + n + k)
    rows = n + 137
    ws = [blocks(mxref.random_blocks(rng, rows, k, 115, 121), k, dev) for _ in range(1 + pair)]
    x, _ = activations(rng, tok, k, kind, dev)
    call = q.qgemv_rows_mx_swiglu if pair else q.qgemv_rows_mx

    def window(r0, r1):
        y = nan_buffer(tok, r1 - r0, "f32", dev)
        call(*ws, r0, r1, x, y)
        return host(y)

    first = window(0, n)
    for r0 in (1, 16, 137):
        assert np.array_equal(window(r0, r0 + n)[:, :n - r0], first[:, r0:]), f"window from {r0}"


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
def test_windows_of_other_sizes(dev, kind):
    rng = np.random.default_rng(4)
    tok, rows, k = 16, 11008, 416
    wb = mxref.random_blocks(rng, rows, k, 115, 121)
    w = blocks(wb, k, dev)
    x, xv = activations(rng, tok, k, kind, dev)
    ref, bound = mxref.product(xv, mxref.values(wb, k), kind)
    for r0, r1 in ((0, rows), (100, 2980), (5, 6), (rows - 33, rows)):
        y = nan_buffer(tok, r1 - r0, "f32", dev)
        q.qgemv_rows_mx(w, r0, r1, x, y)
        mxref.near(host(y), ref[:, r0:r1], bound[:, r0:r1], "f32", f"{r0}..{r1}")


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("tok,n,k", [(40, 60, 416), (700, 523, 224)])
def test_sharing_of_places(dev, kind, pair, tok, n, k):
    """Experts of the same weights: each place's output is the same whichever of them has it."""
    rng = np.random.default_rng(tok + n)
    e = 5
    ws = [blocks(np.tile(mxref.random_blocks(rng, n, k, 115, 121), (e, 1)), k, dev) for _ in range(1 + pair)]
    x, _ = activations(rng, tok, k, kind, dev)
    call = q.qgemv_expert_mx_swiglu if pair else q.qgemv_expert_mx
    got = []
    for cuts in ([0, 0, 0, 0], [tok // 5, 2 * tok // 5, 3 * tok // 5, 4 * tok // 5], [1, 2, tok - 3, tok - 3]):
        y = nan_buffer(tok, n, "f32", dev)
        call(*ws, e, x, dput(np.array([0, *cuts, tok], np.int32), dev), y)
        got.append(host(y))
    assert np.isfinite(got[0]).all()
    assert np.array_equal(got[0], got[1]) and np.array_equal(got[0], got[2])
