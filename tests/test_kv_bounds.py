"""The bounds of kvbound.py on the CPU: the kernels' arithmetic meets them, with one term fewer of q or of the weights,
or with weights or q values that leave most of fp16's range unused, it does not."""
from __future__ import annotations

import pytest
import torch

import kvbound
import kvref
from kvref import TYPES

HEADS, KV, NEW = 4, 2, 24


def over(dim, kind, x, spread, many, **how):
    """Most of its bound that the emulation uses."""
    g = torch.Generator().manual_seed(dim)
    n = 32
    q, (k,), (v,) = kvbound.single(g, [n], NEW, HEADS, KV, dim, kind, x, spread, 8.0)
    seen = kvbound.seen_of(n, NEW)
    ref, _ = kvbound.exact(q, k, v, seen, 8.0)
    t = TYPES[kind]
    top = (7 if many else 15) if kind == "f16" else 0
    got = kvbound.emulated(q, k, v, seen, 8.0, t, **{"q_terms": kvbound.WIDE[t], "w_terms": kvbound.WIDE[t],
                                                    "top_weight": top, "q_top": 14, **how})
    tol = kvbound.bound(ref, v, seen, spread, t, torch.float32, True, many)
    return float(((got.double() - ref).abs() / tol).max())


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("many", [False, True])
def test_bounds_tell_terms_apart(dim, kind, many):
    most = kvbound.WIDE[TYPES[kind]]
    for spread in (1.0, 4.0, 16.0):
        assert over(dim, kind, "f32", spread, many) <= 1.0
    assert over(dim, kind, "f32", 1.0, many, w_terms=most - 1) > 1.2
    assert over(dim, kind, "f32", 4.0, many, q_terms=most - 1) > 1.2
    if kind == "f16":
        assert over(dim, kind, "f32", 16.0, many, top_weight=0) > 1.2
        assert over(dim, kind, "f32", 4.0, many, q_top=0) > 1.2


def test_exact_form_is_the_plain_one():
    g = torch.Generator().manual_seed(3)
    q, (k,), (v,) = kvbound.single(g, [40], 5, HEADS, KV, 32, "f16", "f32", 4.0, 8.0)
    cache = [torch.zeros(1, 3, KV, 16, 32, dtype=torch.float16) for _ in range(2)]
    for c, t in zip(cache, (k, v)):
        for j in range(40):
            c[0, j // 16, :, j % 16] = t[j]
    for causal, window in ((True, 0), (False, 0), (True, 7)):
        ref = kvref.attended(q, [0, 5], [40], torch.arange(3)[None], *cache, 0, 8.0, causal=causal, window=window)
        out, lse = kvbound.exact(q, k, v, kvbound.seen_of(40, 5, causal, window), 8.0)
        assert torch.allclose(out, ref["out"], rtol=1e-12) and torch.allclose(lse, ref["lse"], rtol=1e-12, atol=1e-12)
