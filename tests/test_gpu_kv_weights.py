"""Attention's weights far below their row's largest, over fp16 and bf16 caches: as exact as the type and the terms that
they are taken in allow, few rows and many, whole and cut."""
from __future__ import annotations

import pytest
import torch

import kvref
import quantized_gemv_gguf_amd as q
from kvref import TYPES
from kvsingle import KINDS, check
from test_gpu_kv import ints, within

pytestmark = pytest.mark.gpu

DIMS = [32, 64, 96, 128, 160, 192, 224, 256]


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("dim", DIMS)
def test_weights_apart(dev, dim, kinds):
    """Each output is few weights: relative to it."""
    for spread in (1.0, 16.0):
        check(dev, [32, 20, 7], [1, 2, 3], 4, 2, dim, kinds, spread)
        check(dev, [32, 30], [32, 20], 4, 2, dim, kinds, spread)


@pytest.mark.parametrize("kinds", [KINDS[0], KINDS[2], KINDS[3]])
@pytest.mark.parametrize("dim", [64, 96])
def test_weights_apart_in_parts(dev, dim, kinds):
    """The same of keys that are cut into parts."""
    check(dev, [900], [2], 2, 2, dim, kinds, 16.0, parts=16)
    check(dev, [1500], [40], 2, 2, dim, kinds, 16.0, parts=16)


@pytest.mark.parametrize("x,c,y", [("f32", "f16", "f32"), ("f16", "f16", "f16"), ("f32", "bf16", "f32")])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("above", [8.0, 12.0, 16.0])
def test_one_key_above_many(dev, above, new, x, c, y):
    """One key far above 8191 others, with a value next to theirs of a hundredth: what the others' small weights add."""
    n, dim = 8192 + new - 1, 64
    g = torch.Generator().manual_seed(7)
    k = torch.zeros(1, n // 64 + 1, 1, 64, dim)
    v = 1 + torch.rand(k.shape, generator=g)
    k[..., 0] = torch.rand(k.shape[:-1], generator=g) - 0.5
    k[0, 0, 0, 5], v[0, 0, 0, 5] = 0.0, v[0, 0, 0, 5] / 100
    k[0, 0, 0, 5, 0] = above
    k, v = (t.to(TYPES[c]) for t in (k, v))
    rows = torch.zeros(new, 1, dim)
    rows[..., 0] = 1 + torch.rand(new, 1, generator=g) / 8
    rows = rows.to(TYPES[x])
    cache = q.KvCache(k.to(dev), v.to(dev))
    seqs = q.KvSeqs(ints([0, new], dev), ints([n], dev), torch.arange(k.shape[1], dtype=torch.int32, device=dev)[None])
    xd = rows.to(dev)
    out = torch.empty(new, 1, dim, dtype=TYPES[y], device=dev)
    work = torch.empty(q.qgemv_kv_attend_bytes(xd, seqs, cache), dtype=torch.uint8, device=dev)
    q.qgemv_kv_attend(xd, seqs, cache, 0, out, scale=1.0, work=work)
    table = torch.arange(k.shape[1])[None]
    r = kvref.attended(rows, [0, new], [n], table, k, v, 0, 1.0)
    # scores of at most 18 from one product each: 2^-21 of them, and exp2 and its argument 2^-22; the weights' half-steps
    # (2^-22 of fp16's two terms, 2^-24 of bf16's three).  Sums of positive values: few rows cut the keys into parts of
    # 128, 32 of a wave, 8 of a lane; many into parts of 512, 256 of a lane; then waves and at most 64 parts are joined
    wide = not (x == c == y)
    half = {"f16": 2.0 ** -22, "bf16": 2.0 ** -24}[c] if wide else kvref.EPS[TYPES[c]]
    most_terms = 3 if wide else 1
    sums = 256 + most_terms * 512 if new > 16 else 8 + most_terms * 32
    rel = half + 2 * (18 * 2.0 ** -21 + 2.0 ** -22) + (sums + 2 * 84) * 2.0 ** -24
    lost = {"f16": 2.0 ** -32 if new > 16 else 2.0 ** -40, "bf16": 2.0 ** -120}[c]
    tol = r["out"].abs() * rel + r["total"] * lost
    within(out, r["out"], tol + (r["out"].abs() + tol) * kvref.EPS[TYPES[y]] * 1.001, f"{above} above")
