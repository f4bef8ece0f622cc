"""What the binding of include/qgemv_kv.h refuses on the host (no GPU), and what it passes on."""
from __future__ import annotations

import struct

import pytest

import quantized_gemv_gguf_amd as q

torch = pytest.importorskip("torch")


@pytest.fixture
def on_device(monkeypatch):
    """CPU tensors pass for device tensors; the calls below are refused before any of them is used."""
    q._torch_names()
    monkeypatch.setattr(q, "_current", lambda: 0)
    monkeypatch.setattr(q, "_on", lambda t, dev, name: 0x1000)
    monkeypatch.setattr(q, "_here_stream", lambda stream: 0)


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def cache(kind=torch.float16, layers=1, pages=4, heads=2, size=16, dim=64):
    return q.KvCache(*(torch.zeros(layers, pages, heads, size, dim, dtype=kind) for _ in range(2)))


def seqs(n=1, pages=2):
    return q.KvSeqs(ints(n + 1), ints(n), ints(n, pages))


def pool(n=1, wide=2, pages=4, size=16):
    return q.KvPool(ints(n, wide), ints(n), ints(pages), ints((pages + 31) // 32), size,
                    torch.zeros(q.qgemv_kv_pool_bytes(n, wide, pages), dtype=torch.uint8))


def rope(half=32):
    return q.Rope(torch.zeros(half, dtype=torch.float64))


def test_structs_are_the_headers(on_device):
    """The packed structs lay out the values that the ctypes ones (checked against the header) do."""
    x = torch.zeros(5, 3, 200, dtype=torch.bfloat16)[:, :, 8:72]
    h = q.qg_heads.from_buffer_copy(q._heads(x, 0, "x"))
    assert (h.data, h.type, h.reserved, h.n_tok, h.n_head, h.head_dim, h.tok_stride, h.head_stride) == \
        (0x1000, q.BF16, 0, 5, 3, 64, 600, 200)
    r = q.qg_rope.from_buffer_copy(q._rope(q.Rope(torch.zeros(12, dtype=torch.float64), True, 1.25), 0))
    assert (r.freqs, r.n_rot, r.interleaved, r.mscale) == (0x1000, 24, 1, 1.25)
    c = cache(torch.bfloat16, 3, 5, 2, 16, 96)
    c = q.KvCache(c.k.transpose(2, 3), c.v.transpose(2, 3))
    k = q.qg_kv_cache.from_buffer_copy(q._cache(c, 0))
    assert (k.k, k.v, k.type, k.page_size, k.n_layer, k.n_head, k.head_dim, k.reserved, k.n_pages) == \
        (0x1000, 0x1000, q.BF16, 2, 3, 16, 96, 0, 5)
    assert (k.layer_stride, k.page_stride, k.head_stride, k.slot_stride) == (15360, 3 * 1024, 96, 1536)
    s = q.qg_kv_seqs.from_buffer_copy(q._seqs(seqs(7, 9), 0))
    assert (s.starts, s.lens, s.tables, s.n_seq, s.reserved, s.max_pages) == (0x1000, 0x1000, 0x1000, 7, 0, 9)
    p = q.qg_kv_pool.from_buffer_copy(q._pool(pool(3, 5, 70), 0))
    assert (p.tables, p.lens, p.refs, p.used, p.n_seq, p.page_size, p.max_pages, p.n_pages, p.work) == \
        (0x1000, 0x1000, 0x1000, 0x1000, 3, 16, 5, 70, 0x1000)
    assert p.work_bytes == q.qgemv_kv_pool_bytes(3, 5, 70)
    for packed, of in ((q._HEADS, q.qg_heads), (q._ROPE, q.qg_rope), (q._CACHE, q.qg_kv_cache), (q._SEQS, q.qg_kv_seqs),
                       (q._POOL, q.qg_kv_pool)):
        assert struct.calcsize(packed.format) == len(bytes(of()))


def test_heads(on_device):
    x = torch.zeros(4, 2, 64)
    for bad, error in ((x.double(), TypeError), (x[0], ValueError), (x.transpose(1, 2), ValueError)):
        with pytest.raises(error):
            q.qgemv_rope(bad, ints(4), rope(), x)
        with pytest.raises(error):
            q.qgemv_kv_append(bad, x, seqs(), cache(), 0)
        with pytest.raises(error):
            q.qgemv_kv_attend(x, seqs(), cache(), 0, bad, scale=1.0)
    # heads one value long have no stride of their own
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        q.qgemv_rope(x.transpose(1, 2)[:, :, :1], ints(4), rope(1), x)


def test_arrays(on_device):
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="pos holds 3"):
        q.qgemv_rope(x, ints(3), rope(), x)
    with pytest.raises(TypeError, match="int32"):
        q.qgemv_rope(x, ints(4).long(), rope(), x)
    with pytest.raises(TypeError, match="float64"):
        q.qgemv_rope(x, ints(4), q.Rope(torch.zeros(32)), x)
    with pytest.raises(TypeError, match="float64"):
        q.qgemv_rope(x, ints(4), q.Rope(torch.zeros(64, dtype=torch.float64)[::2]), x)
    for s, name in ((q.KvSeqs(ints(1), ints(1), ints(1, 2)), "starts"), (q.KvSeqs(ints(2), ints(0), ints(1, 2)), "lens")):
        with pytest.raises(ValueError, match=name):
            q.qgemv_kv_attend(x, s, cache(), 0, x, scale=1.0)
    with pytest.raises(ValueError, match="tables must be contiguous"):
        q.qgemv_kv_attend(x, q.KvSeqs(ints(3), ints(2), ints(4, 2).t()[:, :2]), cache(), 0, x, scale=1.0)
    with pytest.raises(ValueError, match="sinks holds 1"):
        q.qgemv_kv_attend(x, seqs(), cache(), 0, x, scale=1.0, sinks=torch.zeros(1))
    with pytest.raises(ValueError, match="lse holds 7"):
        q.qgemv_kv_attend(x, seqs(), cache(), 0, x, scale=1.0, lse=torch.zeros(7))
    with pytest.raises(TypeError, match="lse must be float32"):
        q.qgemv_kv_attend(x, seqs(), cache(), 0, x, scale=1.0, lse=torch.zeros(8).half())
    with pytest.raises(ValueError, match="pos holds 3"):
        q.qgemv_kv_append(x, x, seqs(), cache(), 0, rope=rope(), pos=ints(3))


def test_caches(on_device):
    x, c = torch.zeros(4, 2, 64), cache()
    for bad, error in ((q.KvCache(c.k[0], c.v[0]), ValueError), (q.KvCache(c.k, c.v[:, :3]), ValueError),
                       (q.KvCache(c.k, c.v.bfloat16()), ValueError), (q.KvCache(c.k.int(), c.v.int()), TypeError),
                       (q.KvCache(c.k, c.v.transpose(2, 3).contiguous().transpose(2, 3)), ValueError),
                       (q.KvCache(c.k.transpose(3, 4), c.v.transpose(3, 4)), ValueError)):
        with pytest.raises(error):
            q.qgemv_kv_append(x, x, seqs(), bad, 0)
        with pytest.raises(error):
            q.qgemv_kv_copy(bad, ints(1), ints(1))
    with pytest.raises(q.QgemvError, match="QG_E_FMT"):
        q.qgemv_kv_copy(q.KvCache(c.k.float(), c.v.float()), ints(1), ints(1))
    with pytest.raises(ValueError, match="same length"):
        q.qgemv_kv_copy(c, ints(2), ints(1))


def test_numbers_past_32_bits_are_refused(on_device):
    x = torch.zeros(4, 2, 64)
    with pytest.raises(q.QgemvError, match="QG_E_RANGE"):
        q.qgemv_kv_append(x, x, seqs(), cache(), 1 << 32)
    p = pool()
    p.page_size = (1 << 32) + 16
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        q.qgemv_kv_fork(p, ints(1))
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        q.qgemv_kv_pool_bytes(1 << 32, 1, 1)


def test_workspaces(on_device):
    x = torch.zeros(4, 2, 64)
    wide = seqs(1, 64)
    n = q.qgemv_kv_attend_bytes(x, wide, cache())
    assert n > 0
    for work in (None, torch.zeros(n - 1, dtype=torch.uint8)):
        with pytest.raises(q.QgemvError, match="QG_E_SIZE"):
            q.qgemv_kv_attend(x, wide, cache(), 0, x, scale=1.0, work=work)
    with pytest.raises(ValueError, match="work must be contiguous"):
        q.qgemv_kv_attend(x, wide, cache(), 0, x, scale=1.0, work=torch.zeros(2 * n, dtype=torch.uint8)[::2])
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        q.qgemv_kv_attend_bytes(torch.zeros(4, 3, 64), wide, cache())
    p = pool()
    p.work = p.work[:-1]
    with pytest.raises(q.QgemvError, match="QG_E_SIZE"):
        q.qgemv_kv_fork(p, ints(1))
    with pytest.raises(ValueError, match="parents holds 1"):
        q.qgemv_kv_fork(pool(2), ints(1))
    with pytest.raises(ValueError, match="lens holds 1"):
        q.qgemv_kv_resize(pool(2), cache(), ints(1))


def test_tensors_elsewhere_are_refused(monkeypatch):
    """Host tensors, and tensors of another device than the current one, are named."""
    q._torch_names()
    monkeypatch.setattr(q, "_current", lambda: 0)
    monkeypatch.setattr(q, "_device", lambda: 0)
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        q.qgemv_rope(x, ints(4), rope(), x)

    class Elsewhere:
        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 1

    with pytest.raises(ValueError, match="x is on cuda:1, the current device is cuda:0"):
        q.qgemv_rope(Elsewhere(x), ints(4), rope(), x)
