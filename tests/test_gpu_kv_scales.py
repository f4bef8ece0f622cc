"""Attention over rows of q near fp32's ends, and scales near theirs."""
from __future__ import annotations

import math

import pytest
import torch

from kvsingle import KINDS, check
from test_gpu_kv import Batch, attend, within

pytestmark = pytest.mark.gpu

WIDE = [k for k in KINDS if len(set(k)) > 1]


@pytest.mark.parametrize("kinds", [k for k in WIDE if k[0] != "f16"])
@pytest.mark.parametrize("new", [1, 24])
def test_q_near_the_ends_of_fp32(dev, new, kinds):
    """Rows whose largest value lies in [2^127, 2^128), more than bf16 rounds to a number; and tiny ones, over fp16
    caches subnormal, over bf16 ones with 24 bits above 2^-133; with the scale that belongs to them."""
    check(dev, [32, 32], [new, new], 4, 2, 64, kinds, 4.0, power=127)
    check(dev, [32, 32], [new, new], 4, 2, 64, kinds, 1.0, scale=0.25, power=-129 if kinds[1] == "f16" else -109)


@pytest.mark.parametrize("x,c", [("f32", "f16"), ("bf16", "f16"), ("f32", "bf16")])
@pytest.mark.parametrize("new", [1, 40])
def test_scales_times_q_past_fp32(dev, new, x, c):
    """A scale and a row whose product passes fp32, of keys that are zero: every weight is one."""
    b = Batch(dev, [70], [new], 1, 64, c, seed=3)
    b.k[:] = 0
    b.v.copy_(b.v.abs())
    b.reload()
    q = (torch.randn(new, 2, 64, generator=torch.Generator().manual_seed(1)) * 2.0 ** 30).to(
        torch.float32 if x == "f32" else torch.bfloat16)
    out, lse = attend(b, q, "f32", scale=2.0 ** 110)
    for i in range(new):
        n = 70 - new + i + 1
        v = torch.cat([b.v[1, int(p), 0] for p in b.tables[0, :5]])[:n].double()
        ref = v.mean(0).expand(2, 64)
        within(out[i], ref, ref * (n + 16) * 2.0 ** -24, f"row {i}")
        within(lse[i], torch.full((2,), math.log(n), dtype=torch.float64), torch.full((2,), 2.0 ** -20), f"row {i} lse")
