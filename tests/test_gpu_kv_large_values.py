"""Attention over bf16 values near fp32's end, whose weighted sums are numbers: the running maximum may lag behind the
largest score, which must not make them pass it."""
from __future__ import annotations

import pytest
import torch

from kvref import TYPES
from test_gpu_kv import Batch, attend, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("lens,new", [([300], [1]), ([300, 200], [50, 30]), ([1500], [40])])
def test_large_values_under_rising_scores(dev, lens, new, x, y):
    """The first 64 keys' scores 5 below the others' 0; values of 2^116 to 2^117, so that sums of weights of at most 1
    stay below 2^128 and of e^5 would not."""
    b = Batch(dev, lens, new, 1, 64, "bf16", seed=5)
    g = torch.Generator().manual_seed(6)
    q = torch.zeros(b.rows, 2, 64, dtype=TYPES[x])
    q[..., 0] = 1
    b.k.zero_()
    for s, n in enumerate(lens):
        for j in range(0, 64):
            b.k[1, int(b.tables[s, j // 16]), :, j % 16, 0] = -5.0
    b.v.copy_((1 + torch.rand(b.v.shape, generator=g)) * 2.0 ** 116)
    b.reload()
    out, lse = attend(b, q, y, scale=1.0)
    for s, (n, m) in enumerate(zip(lens, new)):
        at = torch.arange(n)
        v = b.v[1, b.tables[s].long()[at // 16], 0, at % 16].double()
        w = torch.where(at < 64, -5.0, 0.0).double().exp()
        for i in range(m):
            seen = n - m + i + 1
            ref = (w[:seen] @ v[:seen] / w[:seen].sum()).expand(2, 64)
            # weights round once (2^-8; the terms of fp32 rows less), exp2 and sums of n terms beside it
            rel = (2.0 ** -8 if x == y == "bf16" else 2.0 ** -20) + 2 * (n + 64) * 2.0 ** -24
            rel += 2.0 ** -8 if y == "bf16" else 2.0 ** -24
            within(out[b.starts[s] + i], ref, ref * rel * 1.01, f"sequence {s} row {i}")
