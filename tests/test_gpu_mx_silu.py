"""The SiLU of the MXFP4 SwiGLU products (include/qgemv_mx.h) over its range: gate and up rows that pick one value of
x each, so that g and u are exact."""
from __future__ import annotations

import numpy as np
import pytest

import quantized_gemv_gguf_amd as q
from test_gpu_mx import blocks, dput, host, nan_buffer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tok", [3, 1100])
@pytest.mark.parametrize("n", [2, 300])
def test_silu_over_its_range(dev, kind, tok, n):
    rng = np.random.default_rng(tok)
    k = 64
    x = np.zeros((tok, k), np.float32)
    x[:, 0] = rng.uniform(-130, 130, tok)
    x[:3, 0] = [-88.0, -87.0, 0.0]
    x[:, 33] = rng.choice([1.0, -3.0, 1000.0], tok)
    w = np.zeros((2, n, k // 32, 17), np.uint8)
    w[..., 0] = 127
    w[0, :, 0, 1] = 0x02   # 1.0 at element 0
    w[1, :, 1, 2] = 0x02   # 1.0 at element 33
    xd = dput(x, dev, kind)
    y = nan_buffer(tok, n, "f32", dev)
    q.qgemv_rows_mx_swiglu(*[blocks(b.reshape(n, -1), k, dev) for b in w], 0, n, xd, y)
    g, u = host(xd)[:, :1], host(xd)[:, 33:34]
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    # the hardware exp2 and reciprocal cost (|g| + 8) 2^-24 of the value, as in mxref.swiglu; the reciprocal of 2^126 and
    # more is 0, where |silu| is 87.34 * 2^-126 (below 2^-119) and less
    least = np.where(g < -87.3, 2.0 ** -119, 2.0 ** -149)
    assert np.all(np.abs(host(y) - s * u) <= (np.abs(g) + 8) * 2.0 ** -24 * np.abs(s * u) + least * np.abs(u))
