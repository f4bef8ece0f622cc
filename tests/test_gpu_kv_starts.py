"""Attention with starts that do not rise, which gives sequences the same rows: rows and workspace are kept within."""
from __future__ import annotations

import pytest
import torch

import quantized_gemv_gguf_amd as q
from test_gpu_kv import Batch, ints, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [160, 400])
def test_starts_that_do_not_rise(dev, new):
    """More tiles, few rows and many, than the sequences' rows can have: cut into parts whose join stays within them."""
    b = Batch(dev, [3000] * 15, [new] + [0] * 14, 1, 64, "f16", seed=1)
    starts = ints([0, new] * 8, dev)
    x = queries(b, 1, 64, "f16").to(dev)
    seqs = q.KvSeqs(starts, b.seqs.lens, b.seqs.tables)
    n = q.qgemv_kv_attend_bytes(x, seqs, b.cache)
    assert n > 0
    guard = 1 << 20
    work = torch.full((n + guard,), 0x5A, dtype=torch.uint8, device=dev)
    out = torch.full((new + 300, 1, 64), 7.0, dtype=torch.float16, device=dev)
    q.qgemv_kv_attend(x, seqs, b.cache, 1, out[:new], scale=0.3, work=work[:n])
    torch.cuda.synchronize()
    assert (work[n:] == 0x5A).all() and (out[new:] == 7.0).all()
    # the call as it should be, with the same workspace
    q.qgemv_kv_attend(x, b.seqs, b.cache, 1, out[:new], scale=0.3, work=work[:n])
    assert torch.isfinite(out[:new]).all()
