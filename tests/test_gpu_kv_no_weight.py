"""Rows of attention whose every score is -infinity: zeros, whatever the values hold, and the sink's logit or -infinity."""
from __future__ import annotations

import math

import pytest
import torch

from kvref import TYPES
from test_gpu_kv import Batch, attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new", [([100, 7], [1, 2]), ([100, 70], [100, 40]), ([3000], [2]), ([3000], [50])])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_without_weight(dev, causal, lens, new, kind):
    """Few rows and many, whole and cut into parts; one row of each sequence has other scores and is as usual."""
    dim = 64
    b = Batch(dev, lens, new, 1, dim, kind, seed=2)
    b.k[..., 0] = -math.inf
    b.k.nan_to_num_(nan=0.5, neginf=-math.inf)
    q = torch.rand(b.rows, 2, dim, generator=torch.Generator().manual_seed(4)).to(TYPES[kind])
    q[..., 0] += 1
    usual = [r - 1 for r in b.starts[1:]]
    for sizeless in (False, True):
        if sizeless:
            b.v[..., 1], b.v[..., 2], b.v[..., 3] = math.inf, -math.inf, math.nan
            b.v.nan_to_num_(nan=math.nan, posinf=math.inf, neginf=-math.inf)
        b.reload()
        for sinks in (None, torch.tensor([0.25, -3.0])):
            out, lse = attend(b, q, kind, scale=0.5, causal=causal, sinks=sinks)
            assert (out == 0).all(), "not zeros"
            want = torch.full((b.rows, 2), -math.inf) if sinks is None else sinks.expand(b.rows, 2)
            assert torch.allclose(lse.cpu(), want, rtol=2.0 ** -22, atol=0)
    x = q.clone()
    x[usual, :, 0] = 0  # 0 times -infinity: no number, and it stays one
    out, lse = attend(b, x, kind, scale=0.5, causal=causal)
    rest = [r for r in range(b.rows) if r not in usual]
    assert torch.isnan(out[usual]).all() and torch.isnan(lse[usual]).all() and (out[rest] == 0).all()
