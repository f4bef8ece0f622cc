"""GPU parity of the MXFP4 prompt operators (include/qgemv_mx.h) against plain
64-bit forms (mxref.py, where the bounds are derived): quantisation byte for
byte, products within the bound of their fp32 sums, the sort's integers and the
gather bit for bit, and the calls together as a prompt uses them."""
from __future__ import annotations

import numpy as np
import pytest

import mxref
import quantized_gemv_gguf_amd as q
from mxref import near

pytestmark = pytest.mark.gpu


def T(kind):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]


def dput(a, dev, kind=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if kind is None else t.to(T(kind))).to(dev)


def host(t):
    return t.cpu().double().numpy()


def blocks(a, k, dev):
    return q.Matrix(dput(a, dev), q.MXFP4, a.shape[0], k)


def activations(rng, n, k, kind, dev, pad=0):
    """(what the call takes, its values in 64 bits): floats, or MXFP4 blocks."""
    x = rng.standard_normal((n, k + pad)) * 2.0 ** rng.uniform(-3, 3, (1, k + pad))
    if kind == "mxfp4":
        b = mxref.quantize(x[:, :k].astype(np.float32).astype(np.float64))
        return blocks(b, k, dev), mxref.values(b, k)
    t = dput(x.astype(np.float32), dev, kind)[:, :k]
    return t, host(t)


def nan_buffer(n, cols, kind, dev, pad=0):
    import torch
    return torch.full((n, cols + pad), float("nan"), dtype=T(kind), device=dev)


# --- quantisation ------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,pad", [(1, 32, 0), (1, 2880, 0), (3, 64, 5), (257, 96, 1), (70, 4096, 32), (1021, 160, 0)])
def test_quantize(dev, kind, n, k, pad):
    import torch
    rng = np.random.default_rng(n * 1000 + k)
    x = rng.standard_normal((n, k + pad)) * 2.0 ** rng.integers(-6, 6, (n, 1))
    x[0, :8] = [0.25, -0.75, 1.25, 5.0, 6.0, 2.5, 3.5, 0.0]
    if n > 2:
        x[1, :32] = 0.0
        x[2, 3] = np.inf
        x[n - 1, 7] = np.nan
        x[n - 1, 40 % k] = -np.inf
    t = dput(x.astype(np.float32), dev, kind)[:, :k]
    out = torch.full((n * k // 32 * 17 + 64,), 0xA5, dtype=torch.uint8, device=dev)
    m = q.Matrix(out[:n * k // 32 * 17], q.MXFP4, n, k)
    q.qgemv_mx_quantize(t, m)
    ref = mxref.quantize(host(t))
    assert np.array_equal(m.data.cpu().numpy().reshape(n, -1), ref)
    assert (out[n * k // 32 * 17:] == 0xA5).all().item(), "wrote past the blocks"


def test_quantize_range(dev):
    """Every exponent of fp32, subnormals among them, and ties at each of them."""
    import torch
    rows = []
    for e in range(-149, 128):
        s = 2.0 ** max(e - 2, -149)
        r = np.arange(32) * 0.25 * s
        r[31] = 2.0 ** e
        rows.append(np.where(np.arange(32) % 3 == 1, -r, r))
    x = np.array(rows).astype(np.float32)
    m = q.Matrix(torch.zeros(len(rows) * 17, dtype=torch.uint8, device=dev), q.MXFP4, len(rows), 32)
    q.qgemv_mx_quantize(dput(x, dev), m)
    assert np.array_equal(m.data.cpu().numpy().reshape(-1, 17), mxref.quantize(x.astype(np.float64)))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_dequantize_every_code_and_scale(dev, kind):
    import torch
    b = np.zeros((256, 2, 17), np.uint8)
    b[..., 0] = np.arange(256)[:, None]
    b[:, 0, 1:] = np.arange(16) * 17
    b[:, 1, 1:] = (np.arange(16) * 16 + 15 - np.arange(16))
    ref = mxref.values(b.reshape(256, -1), 64)
    out = nan_buffer(250, 64, kind, dev, 3)
    q.qgemv_mx_dequantize(blocks(b.reshape(256, -1), 64, dev), 6, 256, out[:, :64])
    with np.errstate(over="ignore"):
        want = torch.from_numpy(ref[6:]).to(T(kind))
    got = out[:, :64].cpu()
    assert torch.equal(torch.nan_to_num(got.double(), nan=7.0), torch.nan_to_num(want.double(), nan=7.0))
    assert torch.equal(torch.signbit(got)[~torch.isnan(got)], torch.signbit(want)[~torch.isnan(want)])
    assert torch.isnan(out[:, 64:]).all().item()


# --- products ------------------------------------------------------------------------

# tokens, rows, k: single values; one block; tails of the four blocks of a step; rows and tokens around the tiles
SHAPES = [(1, 1, 32), (1, 2880, 2880), (2, 17, 64), (5, 70, 96), (16, 128, 128), (17, 129, 160), (33, 63, 2880),
          (64, 65, 256), (65, 200, 544), (130, 257, 1024), (300, 130, 288), (513, 300, 416), (7, 40, 11008), (16, 8192, 2880)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("tok,n,k", SHAPES)
def test_rows(dev, kind, tok, n, k):
    rng = np.random.default_rng(tok + 7 * n + k)
    out = ["f32", "f16", "bf16"][(tok + n) % 3]
    skip, pad = 3 * (n % 2), n % 5
    wb = mxref.random_blocks(rng, n + skip + 2, k)
    x, xv = activations(rng, tok, k, kind, dev, pad=tok % 4)
    y = nan_buffer(tok, n, out, dev, pad)
    q.qgemv_rows_mx(blocks(wb, k, dev), skip, skip + n, x, y[:, :n])
    ref, bound = mxref.product(xv, mxref.values(wb, k)[skip:skip + n], kind)
    near(host(y[:, :n]), ref, bound, out)
    assert np.isnan(host(y[:, n:])).all(), "wrote past a row"


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("tok,n,k", [(1, 2880, 2880), (3, 33, 96), (18, 64, 544), (100, 190, 256), (260, 129, 416)])
def test_rows_swiglu(dev, kind, tok, n, k):
    rng = np.random.default_rng(tok + n + k)
    out = ["bf16", "f32", "f16"][tok % 3]
    gb, ub = mxref.random_blocks(rng, n + 1, k, 115, 121), mxref.random_blocks(rng, n + 1, k, 115, 121)
    x, xv = activations(rng, tok, k, kind, dev)
    h = nan_buffer(tok, n, out, dev, 1)
    q.qgemv_rows_mx_swiglu(blocks(gb, k, dev), blocks(ub, k, dev), 1, n + 1, x, h[:, :n])
    g, dg = mxref.product(xv, mxref.values(gb, k)[1:], kind)
    u, du = mxref.product(xv, mxref.values(ub, k)[1:], kind)
    near(host(h[:, :n]), *mxref.swiglu(g, dg, u, du), out)
    assert np.isnan(host(h[:, n:])).all()


@pytest.mark.parametrize("tok", [2, 40, 200])
def test_rows_special_values(dev, tok):
    """Scales 255 (NaN) and 0 (subnormal weights), rows of zeros, infinities and NaN of x in their places alone."""
    import torch
    rng = np.random.default_rng(3)
    n, k = 50, 320
    wb = mxref.random_blocks(rng, n, k).reshape(n, -1, 17)
    wb[5, 3, 0] = 255
    wb[20, :, 0] = 0
    # no zero codes where the infinities of x meet them, but in the rows of zeros (whose sums are exactly 0)
    wb[:, 1, 1:] |= 0x11
    wb[30, :, 1:] = 0
    wb[31, :, 1:] = 0x88
    wb = wb.reshape(n, -1)
    wv = mxref.values(wb, k)
    for kind in ("f32", "f16", "bf16"):
        xv = rng.standard_normal((tok, k))
        xv[0, 33], xv[1, 40] = np.inf, np.nan
        x = dput(xv.astype(np.float32), dev, kind)
        if kind == "f32":  # a NaN whose payload is in the lowest bits alone
            x.view(torch.int32)[1, 40] = 0x7f800001
        y = nan_buffer(tok, n, "f32", dev)
        q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, x, y)
        with np.errstate(invalid="ignore"):
            ref, bound = mxref.product(host(x), wv, kind)
        near(host(y), ref, np.where(np.isfinite(bound), bound, 0.0), "f32", kind)
    xb = mxref.random_blocks(rng, tok, k, 120, 128).reshape(tok, -1, 17)
    xb[1, 2, 0] = 255
    xb = xb.reshape(tok, -1)
    y = nan_buffer(tok, n, "f32", dev)
    q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, blocks(xb, k, dev), y)
    ref, bound = mxref.product(mxref.values(xb, k), wv, "mxfp4")
    near(host(y), ref, np.where(np.isfinite(bound), bound, 0.0), "f32", "mxfp4")


def test_rows_f32_keeps_all_bits(dev):
    """x with 24 significant bits against one weight of 1: the exact x comes back (three terms, no rounding)."""
    rng = np.random.default_rng(4)
    k, tok = 64, 40
    wb = np.zeros((k, k // 32, 17), np.uint8)
    wb[..., 0] = 127
    for r in range(k):  # row r picks element r
        e = r % 32
        wb[r, r // 32, 1 + e % 16] = 2 << (4 * (e // 16))
    x = (rng.standard_normal((tok, k)) * 2.0 ** rng.integers(-60, 60, (tok, k))).astype(np.float32)
    for t in (1, 16, tok):
        y = nan_buffer(t, k, "f32", dev)
        q.qgemv_rows_mx(blocks(wb.reshape(k, -1), k, dev), 0, k, dput(x[:t], dev), y)
        assert np.array_equal(host(y), x[:t].astype(np.float64))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tok", [1, 4, 40, 300])
def test_rows_subnormal(dev, kind, tok):
    """Subnormal x, and for float32 normal values whose lower bf16 terms are subnormal, times weights of 2^100: one
    nonzero value of x a token, so that every output is one exact product."""
    rng = np.random.default_rng(tok)
    n, k = 70, 96
    x = np.zeros((tok, k))
    at = rng.integers(0, k, tok)
    low = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}[kind]
    # (bf16 and fp16: as many bits as a subnormal has)
    x[np.arange(tok), at] = low * rng.integers(1, {"f32": 2 ** 24, "f16": 2 ** 10, "bf16": 2 ** 7}[kind], tok)
    wb = mxref.random_blocks(rng, n, k, 227, 228)
    xd = dput(x.astype(np.float32), dev, kind)
    assert np.array_equal(host(xd), x)
    y = nan_buffer(tok, n, "f32", dev)
    q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, xd, y)
    # a 24-bit value times an E2M1 significand (1 or 3): its three terms' products are added with two roundings.
    # bf16's subnormals end at 2^-133, so the float32 terms, which are cut there, leave less than that out of x.
    v = mxref.values(wb, k)
    ref = x @ v.T
    cut = 2.0 ** -133 * np.abs(v[:, at]).T if kind == "f32" else 0.0
    near(host(y), ref, 2.0 ** -23 * np.abs(ref) + cut, "f32")


def test_rows_shared_x_and_no_tokens(dev):
    rng = np.random.default_rng(5)
    n, k = 40, 128
    wb = mxref.random_blocks(rng, n, k)
    x, xv = activations(rng, 1, k, "bf16", dev)
    y = nan_buffer(20, n, "f32", dev)
    q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, x.expand(20, k), y)
    ref, bound = mxref.product(np.repeat(xv, 20, 0), mxref.values(wb, k), "bf16")
    near(host(y), ref, bound, "f32")
    q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, x[:0], y[:0])
    q.qgemv_rows_mx(blocks(wb, k, dev), 9, 9, x.expand(20, k), y[:, :0])
    near(host(y), ref, bound, "f32")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("tok", [1, 3, 33, 70])
def test_rows_largest_k(dev, kind, tok):
    rng = np.random.default_rng(tok)
    n, k = 19, 49152
    wb = mxref.random_blocks(rng, n, k)
    x, xv = activations(rng, tok, k, kind, dev)
    y = nan_buffer(tok, n, "f32", dev)
    q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, x, y)
    ref, bound = mxref.product(xv, mxref.values(wb, k), kind)
    near(host(y), ref, bound, "f32")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tok,n,k", [(2, 40, 96), (50, 300, 224), (300, 520, 160)])
def test_rows_at_odd_addresses(dev, kind, tok, n, k):
    """x and y start one element into their buffers and have odd strides: aligned to one element alone."""
    import torch
    rng = np.random.default_rng(tok)
    wb = mxref.random_blocks(rng, n, k)
    xs, ys = k + 1 + tok % 2, n + 3
    x = torch.zeros(1 + tok * xs, dtype=T(kind), device=dev)
    x.copy_(dput(rng.standard_normal(x.shape).astype(np.float32), dev, kind))
    x = torch.as_strided(x, (tok, k), (xs, 1), 1)
    buf = torch.full((1 + tok * ys,), float("nan"), dtype=T(kind), device=dev)
    y = torch.as_strided(buf, (tok, n), (ys, 1), 1)
    q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, x, y)
    ref, bound = mxref.product(host(x), mxref.values(wb, k), kind)
    near(host(y), ref, bound, kind)
    rest = host(buf)[1:].reshape(tok, ys)[:, n:]
    assert np.isnan(rest).all() and np.isnan(host(buf)[0]), "wrote outside the rows"


# places, rows of W, experts (0: dense): grids large enough for the tiles of many tokens and rows, each kind's
LARGE = [(2049, 130, 0), (700, 1030, 0), (2049, 1030, 0), (2049, 2050, 0), (700, 4100, 0), (65, 8200, 0),
         (200, 8200, 0), (700, 8200, 0), (129, 12300, 0), (200, 12300, 0), (700, 520, 3), (513, 12300, 3),
         (2049, 520, 3), (200, 8200, 8), (2049, 520, 40), (2049, 1030, 40), (90, 1030, 0), (23, 4100, 0), (33, 1030, 8),
         (40, 2050, 3), (129, 2600, 0), (20, 2600, 0), (12, 2600, 0)]


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("places,n,n_expert", LARGE)
def test_large_grids(dev, kind, pair, places, n, n_expert):
    """As test_rows and test_experts; the 64-bit products on the device."""
    import torch
    rng = np.random.default_rng(places + n)
    k, e = (416, 1) if n_expert == 0 else (224, n_expert)
    out = ["bf16", "f32", "f16"][(n + pair) % 3]
    x, xv = activations(rng, places, k, kind, dev)
    wbs = [mxref.random_blocks(rng, e * n, k, 115, 121) for _ in range(1 + pair)]
    ws = [blocks(b, k, dev) for b in wbs]
    y = nan_buffer(places, n, out, dev, 8)
    if n_expert:
        cuts = np.sort(rng.integers(0, places - 20, e - 1))
        offsets = np.concatenate([[0], cuts, [places - 3]])
        call = q.qgemv_expert_mx_swiglu if pair else q.qgemv_expert_mx
        call(*ws, e, x, dput(offsets.astype(np.int32), dev), y[:, :n])
    else:
        offsets = np.array([0, places])
        (q.qgemv_rows_mx_swiglu if pair else q.qgemv_rows_mx)(*ws, 0, n, x, y[:, :n])
    got, xd, kept = y.double(), torch.from_numpy(xv).to(dev), int(offsets[-1])
    assert torch.isnan(got[kept:]).all() and torch.isnan(got[:, n:]).all(), "wrote beyond the places"
    step = 4 * np.ceil(mxref.STEPS[kind] * k) * 2.0 ** -23
    for i in range(e):
        lo, hi = int(offsets[i]), int(offsets[i + 1])
        if lo == hi:
            continue
        r = []
        for b in wbs:
            w = torch.from_numpy(mxref.values(b[i * n:(i + 1) * n], k)).to(dev)
            r.append((xd[lo:hi] @ w.T, step * (xd[lo:hi].abs() @ w.abs().T)))
        ref, bound = r[0]
        if pair:
            (g, dg), (u, du) = r
            silu = g / (1 + torch.exp(-g))
            ref = silu * u
            bound = 1.1 * dg * (u.abs() + du) + silu.abs() * du + (g.abs() + 8) * 2.0 ** -24 * ref.abs()
        err = (got[lo:hi, :n] - ref).abs()
        allowed = bound + mxref.HALF[out] * (ref.abs() + bound) + mxref.TINY[out]
        assert bool((err <= allowed).all()), f"expert {i}: worst {float((err / allowed).max()):.3g} times the bound"


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_large_gathered(dev, kind, pair, out):
    """Tiles of many tokens that gather x through slots: tokens named more than once, slots of tokens that x does not
    have (rows of zeros), an expert without a place, offsets below zero and beyond the places."""
    import torch
    rng = np.random.default_rng(21)
    tok, sel, places, n, k, e = 700, 2, 2049, 523, 160, 3
    x, xv = activations(rng, tok, k, kind, dev)
    wbs = [mxref.random_blocks(rng, e * n, k, 117, 121) for _ in range(1 + pair)]
    slots = rng.integers(0, sel * tok, places)
    foreign = rng.choice(places, 40, replace=False)
    slots[foreign] = rng.choice([-1, -2 ** 31, sel * tok, 2 ** 31 - 1], 40)
    call = q.qgemv_expert_mx_swiglu if pair else q.qgemv_expert_mx
    y = nan_buffer(places, n, out, dev, 3)
    call(*[blocks(b, k, dev) for b in wbs], e, x, dput(np.array([-7, 600, 600, 5000], np.int32), dev), y[:, :n],
         slots=dput(slots.astype(np.int32), dev), n_sel=sel)
    xs = xv[np.clip(slots // sel, 0, tok - 1)]
    xs[foreign] = 0
    got = host(y)
    assert np.isnan(got[:, n:]).all()
    for i, lo, hi in ((0, 0, 600), (2, 600, places)):
        r = [mxref.product(xs[lo:hi], mxref.values(b[i * n:(i + 1) * n], k), kind) for b in wbs]
        ref, bound = mxref.swiglu(*r[0], *r[1]) if pair else r[0]
        near(got[lo:hi, :n], ref, bound, out)


def test_offsets_past_32_bits(dev):
    """Rows of x and y gigabytes apart, and a stack of experts above 4 GiB."""
    import torch
    rng = np.random.default_rng(12)
    n, k, tok, apart = 70, 96, 40, (1 << 26) + 8
    wb = mxref.random_blocks(rng, n, k)
    xbuf = torch.empty(tok * apart, dtype=torch.bfloat16, device=dev)
    ybuf = torch.empty(tok * apart, dtype=torch.bfloat16, device=dev)
    x, y = torch.as_strided(xbuf, (tok, k), (apart, 1)), torch.as_strided(ybuf, (tok, n), (apart, 1))
    x.copy_(dput(rng.standard_normal((tok, k)).astype(np.float32), dev, "bf16"))
    q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, x, y)
    ref, bound = mxref.product(host(x), mxref.values(wb, k), "bf16")
    near(host(y), ref, bound, "bf16")
    out = torch.empty_like(x.contiguous())
    q.qgemv_expert_gather(x, torch.arange(tok, dtype=torch.int32, device=dev), 1, out)
    assert torch.equal(out, x)
    back = torch.as_strided(ybuf, (tok, k), (apart, 1))
    q.qgemv_expert_combine(x, torch.arange(tok, dtype=torch.int32, device=dev).view(tok, 1), back)
    assert torch.equal(back, x)
    del xbuf, ybuf, x, y, out, back
    n_expert, n, k = 1024, 2880, 2880
    w = torch.randint(0, 256, (n_expert * n, k // 32 * 17), dtype=torch.uint8, device=dev)
    w[:, ::17] = 118
    assert w.numel() > 1 << 32
    tok = 30
    offsets = torch.full((n_expert + 1,), tok, dtype=torch.int32, device=dev)
    offsets[0], offsets[1:n_expert] = 0, 7   # seven tokens at the first expert, the others at the last
    x = torch.randn(tok, k, device=dev)
    y = nan_buffer(tok, n, "f32", dev)
    q.qgemv_expert_mx(q.Matrix(w, q.MXFP4, n_expert * n, k), n_expert, x, offsets, y)
    for lo, hi, e in ((0, 7, 0), (7, tok, n_expert - 1)):
        ref, bound = mxref.product(host(x[lo:hi]), mxref.values(w[e * n:(e + 1) * n].cpu().numpy(), k), "f32")
        near(host(y[lo:hi]), ref, bound, "f32")


def test_more_workgroups_than_a_grid(dev):
    """Calls whose threads one launch does not hold (2^32 and more of them)."""
    import torch

    def ones(rows, cols, e):  # every code 1.0, scale e
        w = torch.full((rows, cols // 32 * 17), 0x22, dtype=torch.uint8, device=dev)
        w[:, ::17] = e
        return q.Matrix(w, q.MXFP4, rows, cols)

    # one token, 2^29 + 3 rows of one block
    n = 2 ** 29 + 3
    w = ones(n, 32, 127)
    w.data[n - 1, 0], w.data[2 ** 29 - 1, 0] = 128, 126
    y = torch.full((1, n), -1.0, dtype=torch.bfloat16, device=dev)
    q.qgemv_rows_mx(w, 0, n, torch.ones(1, 32, device=dev), y)
    assert y[0, n - 1] == 64 and y[0, 2 ** 29 - 1] == 16
    y[0, n - 1] = y[0, 2 ** 29 - 1] = 32
    assert bool((y == 32).all())
    del w, y
    torch.cuda.empty_cache()
    # 2^30 + 96 blocks back
    n, k = 2 ** 15 + 1, 2 ** 15
    w = ones(n, k, 127)
    w.data[n - 1, ::17] = 130
    out = torch.zeros(n, k, dtype=torch.bfloat16, device=dev)
    q.qgemv_mx_dequantize(w, 0, n, out)
    assert bool((out[:n - 1] == 1).all()) and bool((out[n - 1] == 8).all())
    # ... and 2^32 + 2^17 of them from a row that is repeated
    del w, out
    torch.cuda.empty_cache()
    n, k = 2 ** 22 + 128, 2 ** 15
    x = torch.full((1, k), 3.0, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(n, k // 32 * 17, dtype=torch.uint8, device=dev)
    q.qgemv_mx_quantize(x.expand(n, k), q.Matrix(w, q.MXFP4, n, k))
    for lo in range(0, n, 2 ** 19):
        part = w[lo:lo + 2 ** 19].view(-1, 17)
        assert bool((part[:, 0] == 126).all()) and bool((part[:, 1:] == 0x77).all())
    del w, part
    torch.cuda.empty_cache()
    # 2^25 tokens of a row of 513: 128 threads each
    n, cols = 2 ** 25 + 5, 513
    y = torch.full((4, cols), 2.0, dtype=torch.bfloat16, device=dev)
    out = torch.zeros(n, cols, dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(n, 1, dtype=torch.int32, device=dev)
    pos[n - 1] = -1
    out[n - 1] = 7
    q.qgemv_expert_combine(y, pos, out)
    assert bool((out[:n - 1] == 2).all()) and bool((out[n - 1] == 0).all())
    del out
    torch.cuda.empty_cache()
    # 2^24 slots of a workgroup each, two of them kept
    n = 2 ** 24 + 9
    pos = torch.full((n, 1), -1, dtype=torch.int32, device=dev)
    pos[1], pos[n - 2] = 0, 3
    wts = torch.full((n, 1), 3.0, device=dev)
    dw = torch.full((n, 1), -1.0, device=dev)
    dy = torch.full_like(y, 5.0)
    q.qgemv_expert_combine_grad(y[:1].expand(n, cols), y, pos, wts, dy, dw)
    assert bool((dy[0] == 6).all()) and bool((dy[1:3] == 5).all()) and bool((dy[3] == 6).all())
    assert dw[1] == 4 * cols and dw[n - 2] == 4 * cols
    dw[1] = dw[n - 2] = 0
    assert not dw.any()
    torch.cuda.empty_cache()


def test_quantize_past_32_bits(dev):
    import torch
    n, k = (1 << 26) + 3, 96  # 6.4 billion values, 3.4 GB of blocks
    x = torch.empty(n, k, dtype=torch.bfloat16, device=dev).normal_()
    m = q.Matrix(torch.empty(n * k // 32 * 17, dtype=torch.uint8, device=dev), q.MXFP4, n, k)
    q.qgemv_mx_quantize(x, m)
    back = torch.empty_like(x)
    q.qgemv_mx_dequantize(m, 0, n, back)
    for r in (0, 12345, n // 2, n - 5):
        b = m.data.view(n, -1)[r:r + 5].cpu().numpy()
        assert np.array_equal(b, mxref.quantize(host(x[r:r + 5])))
        assert np.array_equal(host(back[r:r + 5]), mxref.values(b, k))


# --- experts ---------------------------------------------------------------------------

def expert_case(rng, tok, sel, n_expert, dropped):
    ids = np.stack([rng.permutation(max(n_expert, sel))[:sel] for _ in range(tok)]).reshape(tok, sel)
    ids[rng.random((tok, sel)) < dropped] = -1
    return ids


# tokens, choices, experts, rows, k, share of dropped slots
EXPERTS = [(1, 1, 1, 16, 32, 0.0), (1, 4, 128, 96, 160, 0.0), (3, 2, 5, 33, 96, 0.2), (40, 4, 16, 130, 288, 0.1),
           (200, 2, 3, 70, 256, 0.0), (130, 8, 64, 64, 128, 0.3), (64, 1, 200, 20, 64, 0.0), (9, 3, 4, 40, 64, 1.0),
           (70, 2, 1024, 5, 32, 0.0), (500, 2, 7, 65, 160, 0.05)]


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("tok,sel,n_expert,n,k,dropped", EXPERTS)
def test_experts(dev, kind, pair, tok, sel, n_expert, n, k, dropped):
    rng = np.random.default_rng(tok * sel + n_expert + n)
    out = ["f32", "bf16", "f16"][(tok + pair) % 3]
    ids = expert_case(rng, tok, sel, n_expert, dropped)
    offsets, slots, _ = mxref.sort(ids, n_expert)
    gathered = (n + k // 32) % 2 == 0
    spare = 3  # places behind the last slot
    x, xv = activations(rng, tok if gathered else tok * sel + spare, k, kind, dev)
    wbs = [mxref.random_blocks(rng, n_expert * n, k, 115, 121) for _ in range(1 + pair)]
    y = nan_buffer(tok * sel + spare, n, out, dev, 2)
    sl = dput(np.concatenate([slots, [-1] * spare]).astype(np.int32), dev)
    call = q.qgemv_expert_mx_swiglu if pair else q.qgemv_expert_mx
    call(*[blocks(b, k, dev) for b in wbs], n_expert, x, dput(offsets.astype(np.int32), dev), y[:, :n],
         **(dict(slots=sl, n_sel=sel) if gathered else {}))
    got = host(y)
    kept = offsets[-1]
    assert np.isnan(got[kept:]).all() and np.isnan(got[:, n:]).all(), "wrote beyond the places"
    for e in range(n_expert):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        xs = xv[slots[lo:hi] // sel] if gathered else xv[lo:hi]
        r = [mxref.product(xs, mxref.values(b[e * n:(e + 1) * n], k), kind) for b in wbs]
        near(got[lo:hi, :n], *(mxref.swiglu(*r[0], *r[1]) if pair else r[0]), out, f"expert {e}")


def test_experts_all_to_one_and_foreign_slots(dev):
    """Every token at the last expert; slots that name tokens x does not have count as rows of zeros."""
    import torch
    rng = np.random.default_rng(8)
    tok, n_expert, n, k = 150, 12, 48, 192
    x, xv = activations(rng, tok, k, "bf16", dev)
    wb = mxref.random_blocks(rng, n_expert * n, k)
    offsets = torch.zeros(n_expert + 1, dtype=torch.int32, device=dev)
    offsets[-1] = tok
    slots = torch.arange(tok, dtype=torch.int32, device=dev)
    slots[7], slots[149] = tok + 5, -3
    y = nan_buffer(tok, n, "f32", dev)
    q.qgemv_expert_mx(blocks(wb, k, dev), n_expert, x, offsets, y, slots=slots, n_sel=1)
    xv = xv.copy()
    xv[[7, 149]] = 0
    ref, bound = mxref.product(xv, mxref.values(wb[-n:], k), "bf16")
    near(host(y), ref, bound, "f32")
    # offsets beyond the places are clamped to them
    offsets[-1] = tok + 1000
    y.fill_(float("nan"))
    q.qgemv_expert_mx(blocks(wb, k, dev), n_expert, x, offsets, y, slots=slots, n_sel=1)
    near(host(y), ref, bound, "f32")


# --- routing ---------------------------------------------------------------------------

@pytest.mark.parametrize("tok,sel,n_expert,dropped", [(0, 4, 8, 0.0), (1, 1, 1, 0.0), (1, 4, 128, 0.0), (63, 1, 2, 0.3),
                                                      (64, 4, 16, 0.0), (65, 4, 1024, 0.1), (257, 8, 60, 0.5),
                                                      (1500, 4, 128, 0.02), (3000, 6, 7, 0.0), (5, 2, 3, 1.0)])
def test_sort(dev, tok, sel, n_expert, dropped):
    import torch
    rng = np.random.default_rng(tok + sel)
    ids = rng.integers(0, n_expert, (tok, sel))
    out = rng.random((tok, sel)) < dropped
    ids[out] = rng.choice([-1, -2 ** 31, n_expert, 2 ** 31 - 1], out.sum())
    n = tok * sel
    bufs = [torch.full((m + 4,), 77, dtype=torch.int32, device=dev) for m in (n_expert + 1, n, n)]
    q.qgemv_expert_sort(dput(ids.astype(np.int32), dev).view(tok, sel), n_expert, *bufs)
    for buf, ref in zip(bufs, mxref.sort(ids, n_expert)):
        assert np.array_equal(buf.cpu().numpy(), np.concatenate([ref.ravel(), [77] * 4]))


@pytest.mark.parametrize("tok,sel,n_expert,dropped", [(65536, 1, 16, 0.1), (65537, 1, 16, 0.1), (16385, 4, 128, 0.0),
                                                      (70001, 1, 1024, 0.3), (40000, 2, 1, 0.5), (33000, 2, 1000, 1.0),
                                                      (21900, 3, 7, 0.02), (150001, 8, 60, 0.0), (300000, 4, 129, 0.01),
                                                      (4096, 4, 1024, 0.1), (4097, 4, 1024, 0.1), (6554, 5, 257, 0.0)])
def test_sort_many_slots(dev, tok, sel, n_expert, dropped):
    """As test_sort, around and above the size from which chunks of slots are sorted in several launches; twice."""
    import torch
    rng = np.random.default_rng(tok + sel)
    ids = np.minimum((n_expert * rng.random(tok * sel) ** 2).astype(np.int64), n_expert - 1)   # uneven
    out = rng.random(tok * sel) < dropped
    ids[out] = rng.choice([-1, -2 ** 31, n_expert, 2 ** 31 - 1], out.sum())
    n, kept = tok * sel, (ids >= 0) & (ids < n_expert)
    order = np.argsort(np.where(kept, ids, n_expert), kind="stable")
    slots, pos = np.where(np.arange(n) < kept.sum(), order, -1), np.full(n, -1)
    pos[order[:kept.sum()]] = np.arange(kept.sum())
    offsets = np.searchsorted(ids[order[:kept.sum()]], np.arange(n_expert + 1))
    bufs = [torch.full((m + 4,), 77, dtype=torch.int32, device=dev) for m in (n_expert + 1, n, n)]
    for _ in range(2):
        q.qgemv_expert_sort(dput(ids.astype(np.int32), dev).view(tok, sel), n_expert, *bufs)
        for buf, ref in zip(bufs, (offsets, slots, pos)):
            assert np.array_equal(buf.cpu().numpy(), np.concatenate([ref, [77] * 4]))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tok,sel,cols", [(1, 4, 2880), (5, 1, 1), (9, 2, 7), (33, 3, 64), (40, 4, 250), (20, 2, 2049)])
def test_gather(dev, kind, tok, sel, cols):
    import torch
    rng = np.random.default_rng(cols)
    x = dput(rng.standard_normal((tok, cols + 3)).astype(np.float32), dev, kind)[:, :cols]
    slots = rng.permutation(tok * sel).astype(np.int32)
    slots[::5] = -1
    slots[1::7] = tok * sel + 9
    out = nan_buffer(tok * sel, cols, kind, dev, 1)
    q.qgemv_expert_gather(x, dput(slots, dev), sel, out[:, :cols])
    ok = (slots >= 0) & (slots < tok * sel)
    got = out.cpu()
    assert torch.equal(got[ok][:, :cols], x.cpu()[slots[ok] // sel])
    assert torch.isnan(got[~ok]).all() and torch.isnan(got[:, cols:]).all()


@pytest.mark.parametrize("ky,ko", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("tok,sel,cols", [(1, 4, 2880), (5, 1, 1), (9, 2, 7), (33, 3, 64), (12, 8, 4100), (3, 0, 40)])
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(dev, ky, ko, tok, sel, cols, weighted):
    import torch
    rng = np.random.default_rng(cols + sel)
    rows = max(1, tok * sel)
    y = dput(rng.standard_normal((rows, cols + 2)).astype(np.float32), dev, ky)[:, :cols]
    pos = rng.permutation(rows)[:tok * sel].reshape(tok, sel)
    pos[rng.random((tok, sel)) < 0.2] = -1
    if sel:
        pos[0] = -1          # a token without any expert
        pos[-1, 0] = rows    # beyond y
    w = rng.standard_normal((tok, sel)).astype(np.float32)
    out = nan_buffer(tok, cols, ko, dev, 3)
    q.qgemv_expert_combine(y, dput(pos.astype(np.int32), dev), out[:, :cols], w=dput(w, dev) if weighted else None)
    yv, ref, mag = host(y), np.zeros((tok, cols)), np.zeros((tok, cols))
    for t in range(tok):
        for s in range(sel):
            if 0 <= pos[t, s] < rows:
                term = (float(w[t, s]) if weighted else 1.0) * yv[pos[t, s]]
                ref[t] += term
                mag[t] += np.abs(term)
    near(host(out[:, :cols]), ref, sel * 2.0 ** -24 * mag, ko)
    assert np.isnan(host(out[:, cols:])).all()


@pytest.mark.parametrize("kd,ky", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("tok,sel,cols", [(1, 4, 2880), (5, 1, 1), (9, 2, 7), (33, 3, 64), (6, 8, 4100)])
def test_combine_grad(dev, kd, ky, tok, sel, cols):
    import torch
    rng = np.random.default_rng(cols + sel)
    rows = tok * sel
    dout = dput(rng.standard_normal((tok, cols)).astype(np.float32), dev, kd)
    y = dput(rng.standard_normal((rows, cols + 2)).astype(np.float32), dev, ky)[:, :cols]
    pos = rng.permutation(rows).reshape(tok, sel)
    pos[rng.random((tok, sel)) < 0.2] = -1
    w = rng.standard_normal((tok, sel)).astype(np.float32)
    dy = nan_buffer(rows, cols, ky, dev, 1)
    dw = torch.full((tok, sel), float("nan"), device=dev)
    q.qgemv_expert_combine_grad(dout, y, dput(pos.astype(np.int32), dev), dput(w, dev), dy[:, :cols], dw)
    dv, yv, got, gw = host(dout), host(y), host(dy), host(dw)
    named = np.zeros(rows, bool)
    for t in range(tok):
        for s in range(sel):
            p = pos[t, s]
            if p < 0:
                assert gw[t, s] == 0.0
                continue
            named[p] = True
            near(got[p, :cols], float(w[t, s]) * dv[t], 0.0, ky)
            # a lane's run of fmas, six additions over the lanes and two over the waves
            adds = 8 * -(-cols // 2048) + 8
            mag = np.sum(np.abs(dv[t] * yv[p]))
            near(gw[t, s:s + 1], np.sum(dv[t] * yv[p])[None], adds * 2.0 ** -24 * mag, "f32")
    assert np.isnan(got[~named]).all() and np.isnan(got[:, cols:]).all()


# --- together ----------------------------------------------------------------------------

class Block:
    """A mixture of experts: its weights, a prompt, and the calls of one pass."""

    def __init__(self, dev, tok, sel, n_expert, d, f, kind="bf16", four_bit=False, dropped=0.1, seed=1):
        import torch
        rng = np.random.default_rng(seed)
        self.n_expert, self.sel, self.four_bit, self.kind = n_expert, sel, four_bit, kind
        self.ids_host = expert_case(rng, tok, sel, n_expert, dropped)
        self.wb = [mxref.random_blocks(rng, n_expert * n, k, 115, 121) for n, k in ((f, d), (f, d), (d, f))]
        self.w = [blocks(b, k, dev) for b, k in zip(self.wb, (d, d, f))]
        self.x, self.xv = activations(rng, tok, d, kind, dev)
        self.rw_host = rng.random((tok, sel)).astype(np.float32)
        self.ids, self.rw = dput(self.ids_host.astype(np.int32), dev), dput(self.rw_host, dev)
        z = lambda n, t: torch.zeros(n, dtype=t, device=dev)  # noqa: E731
        self.offsets, self.slots, self.pos = z(n_expert + 1, torch.int32), z(tok * sel, torch.int32), z((tok, sel), torch.int32)
        self.h, self.y = z((tok * sel, f), T(kind)), z((tok * sel, d), T(kind))
        self.out = z((tok, d), torch.float32)
        self.xq = q.Matrix(z(tok * d // 32 * 17, torch.uint8), q.MXFP4, tok, d)
        self.hq = q.Matrix(z(tok * sel * f // 32 * 17, torch.uint8), q.MXFP4, tok * sel, f)

    def run(self, stream=None):
        x, h = self.x, self.h
        q.qgemv_expert_sort(self.ids, self.n_expert, self.offsets, self.slots, self.pos, stream=stream)
        if self.four_bit:
            q.qgemv_mx_quantize(x, self.xq, stream=stream)
            x = self.xq
        q.qgemv_expert_mx_swiglu(*self.w[:2], self.n_expert, x, self.offsets, self.h, slots=self.slots,
                                 n_sel=self.sel, stream=stream)
        if self.four_bit:
            q.qgemv_mx_quantize(h, self.hq, stream=stream)
            h = self.hq
        q.qgemv_expert_mx(self.w[2], self.n_expert, h, self.offsets, self.y, stream=stream)
        q.qgemv_expert_combine(self.y, self.pos, self.out, w=self.rw, stream=stream)
        return self.out


@pytest.mark.parametrize("tok,four_bit", [(1, False), (37, False), (37, True), (300, False), (300, True)])
def test_a_prompt_through_the_experts(dev, tok, four_bit):
    """Every stage against its definition on the stage before, as computed."""
    b = Block(dev, tok, 4, 16, 160, 96, four_bit=four_bit)
    b.run()
    offsets, slots, pos = mxref.sort(b.ids_host, b.n_expert)
    assert np.array_equal(b.pos.cpu().numpy(), pos)
    kept = offsets[-1]
    kind = "mxfp4" if four_bit else b.kind
    xv = mxref.values(mxref.quantize(b.xv), 160) if four_bit else b.xv
    hv, yv = host(b.h)[:kept], host(b.y)[:kept]
    hin = mxref.values(mxref.quantize(hv), 96) if four_bit else hv
    for e in range(b.n_expert):
        lo, hi = offsets[e], offsets[e + 1]
        xs = xv[slots[lo:hi] // 4]
        g, u = (mxref.product(xs, mxref.values(wb[e * 96:(e + 1) * 96], 160), kind) for wb in b.wb[:2])
        near(hv[lo:hi], *mxref.swiglu(*g, *u), b.kind)
        near(yv[lo:hi], *mxref.product(hin[lo:hi], mxref.values(b.wb[2][e * 160:(e + 1) * 160], 96), kind), b.kind)
    ref, mag = np.zeros((tok, 160)), np.zeros((tok, 160))
    for t in range(tok):
        for s in range(4):
            if pos[t, s] >= 0:
                ref[t] += b.rw_host[t, s].astype(np.float64) * yv[pos[t, s]]
                mag[t] += np.abs(b.rw_host[t, s].astype(np.float64) * yv[pos[t, s]])
    near(host(b.out), ref, 4 * 2.0 ** -24 * mag, "f32")


def test_captured_replayed_and_on_other_streams(dev):
    """The pass captured once and replayed on new inputs, each replay against the eager pass, eager work between
    them; and two passes at once on two streams."""
    import torch
    a, b = Block(dev, 90, 4, 16, 160, 96, seed=2), Block(dev, 70, 2, 9, 128, 64, "f32", seed=3)
    want_a, want_b = a.run().clone(), b.run().clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.out.zero_(), b.out.zero_()
        torch.cuda.synchronize()
        a.run(s1), b.run(s2)
        torch.cuda.synchronize()
        assert torch.equal(a.out, want_a) and torch.equal(b.out, want_b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    rng = np.random.default_rng(9)
    for i in range(4):
        a.x.copy_(dput(rng.standard_normal(a.x.shape).astype(np.float32), dev, "bf16"))
        a.ids.copy_(dput(expert_case(rng, 90, 4, 16, 0.1 * i).astype(np.int32), dev))
        g.replay()
        torch.cuda.synchronize()
        got = a.out.clone()
        a.out.zero_()
        assert torch.equal(a.run(), got)


@pytest.mark.parametrize("tok,sel,cols", [(7, 3, 45), (16, 2, 64)])
def test_gradients_against_differences(dev, tok, sel, cols):
    """<dout, combine> moved along random directions of y and w, and <dxs, gather> along x: both are linear in each
    argument, so the difference is the directional derivative up to fp32 rounding."""
    import torch
    rng = np.random.default_rng(11)
    ids = expert_case(rng, tok, sel, 5, 0.2)
    offsets, slots, pos = mxref.sort(ids, 5)
    P, S = dput(pos.astype(np.int32), dev), dput(slots.astype(np.int32), dev)
    r = lambda *s: dput(rng.standard_normal(s).astype(np.float32), dev)  # noqa: E731
    y, w, dout, ydir, wdir = r(tok * sel, cols), r(tok, sel), r(tok, cols), r(tok * sel, cols), r(tok, sel)
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    q.qgemv_expert_combine_grad(dout, y, P, w, dy, dw)

    def loss(yy, ww):
        out = torch.empty(tok, cols, device=dev)
        q.qgemv_expert_combine(yy, P, out, w=ww)
        return float((out.double() * dout.double()).sum())

    # n terms of magnitude about 1 each, fp32 sums within: n * sel * 2^-24 and the inputs' own rounding
    tol = 8 * (sel + 4) * 2.0 ** -24 * tok * cols * sel
    assert abs((loss(y + ydir, w) - loss(y, w)) - float((dy.double() * ydir.double()).sum())) <= tol
    assert abs((loss(y, w + wdir) - loss(y, w)) - float((dw.double() * wdir.double()).sum())) <= tol
    x, xdir, dxs = r(tok, cols), r(tok, cols), r(tok * sel, cols)
    dx = torch.empty(tok, cols, device=dev)
    q.qgemv_expert_combine(dxs, P, dx)

    def gathered(v):
        out = torch.zeros(tok * sel, cols, device=dev)
        q.qgemv_expert_gather(v, S, sel, out)
        return float((out.double() * dxs.double()).sum())

    assert abs((gathered(x + xdir) - gathered(x)) - float((dx.double() * xdir.double()).sum())) <= tol


def test_refusals_leave_outputs(dev):
    import torch
    w = blocks(mxref.random_blocks(np.random.default_rng(1), 8, 64), 64, dev)
    x = torch.ones(4, 64, device=dev)
    y = torch.full((4, 8), 7.0, device=dev)
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        q.qgemv_rows_mx(w, 0, 7, x, y)
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        q.qgemv_rows_mx(w, 0, 8, x[:3], y)
    with pytest.raises(q.QgemvError, match="QG_E_FMT"):
        q.qgemv_rows_mx(q.Matrix(torch.zeros(8 * 2 * 18, dtype=torch.uint8, device=dev), q.Q4_0, 8, 64), 0, 8, x, y)
    with pytest.raises(q.QgemvError, match="QG_E_ARG"):
        q.qgemv_rows_mx(w, 0, 8, x, y[:1].expand(4, 8))
    with pytest.raises(ValueError, match="needs"):
        q.qgemv_expert_mx(w, 2, x, torch.zeros(2, dtype=torch.int32, device=dev), y[:, :4].contiguous())
    with pytest.raises(ValueError, match="needs"):
        q.qgemv_rows_mx(w, 0, 8, q.Matrix(torch.zeros(17, dtype=torch.uint8, device=dev), q.MXFP4, 4, 64), y)
    assert (y == 7.0).all().item()
