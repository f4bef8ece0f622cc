"""MXFP4 products (include/qgemv_mx.h) over the largest scale bytes, 250 to 254:
codes 2, 3, 4 and 6 at 254 and 4 and 6 at 253 are weights of 2^128 and more,
which neither bf16 nor fp32 holds, while their products with small x are
ordinary numbers and with zeros are zero."""
from __future__ import annotations

import numpy as np
import pytest

import mxref
import quantized_gemv_gguf_amd as q
from mxref import near
from test_gpu_mx import blocks, dput, host, nan_buffer

pytestmark = pytest.mark.gpu


def huge_weights(rng, n, k, rows):
    """Ordinary blocks, but one of scale 250 .. 254 in each of `rows` (never a row's first block)."""
    b = mxref.random_blocks(rng, n, k, 115, 121).reshape(n, k // 32, 17)
    for j, r in enumerate(rows):
        b[r, 1 + rng.integers(k // 32 - 1), 0] = 250 + j % 5
    return b.reshape(n, -1)


def small_tokens(rng, tok, k, kind, single):
    """Tokens in turn: zero but in the first block; tiny; small; and (single) one value of 0.5 or 1 beyond the first
    block."""
    x = rng.standard_normal((tok, k))
    first = np.arange(k) < 32
    tiny = 2.0 ** (-14 if kind == "f16" else -100)
    for t in range(tok):
        if t % 4 in (0, 3):
            x[t, ~first] = 0.0
        else:
            x[t] *= tiny if t % 4 == 1 else 2.0 ** -12
        if single and t % 4 == 3:
            x[t, rng.integers(32, k)] = rng.choice([0.5, 1.0])
    return x


def as_given(x, kind, dev):
    if kind == "mxfp4":
        b = mxref.quantize(x.astype(np.float32).astype(np.float64))
        return blocks(b, x.shape[1], dev), mxref.values(b, x.shape[1])
    t = dput(x.astype(np.float32), dev, kind)
    return t, host(t)


def past_range(ref):
    """fp32's infinities; the products here keep well away from half a step below 2^128."""
    return np.where(np.abs(ref) >= 2.0 ** 128 - 2.0 ** 103, np.copysign(np.inf, ref), ref)


def check_huge(dev, kind, pair, tok, n, k, out="f32", n_expert=0):
    """Dense, or in `n_expert` equal runs of tokens gathered through slots, with one slot that x does not have."""
    rng = np.random.default_rng(tok + n + k)
    e = max(n_expert, 1)
    rows = np.arange(0, e * n, 7)
    wbs = [huge_weights(rng, e * n, k, (rows + 3 * i) % (e * n)) for i in range(1 + pair)]
    wbs[0][-1] = huge_weights(rng, 1, k, [0, 0, 0, 0, 0])
    x, xv = as_given(small_tokens(rng, tok, k, kind, not pair), kind, dev)
    y = nan_buffer(tok, n, out, dev, 1)
    ws = [blocks(b, k, dev) for b in wbs]
    offsets = np.linspace(0, tok, e + 1).astype(np.int32)
    if n_expert:
        slots = np.arange(tok, dtype=np.int32)
        slots[tok // 2] = tok
        xv = xv.copy()
        xv[tok // 2] = 0.0
        (q.qgemv_expert_mx_swiglu if pair else q.qgemv_expert_mx)(*ws, e, x, dput(offsets, dev), y[:, :n],
                                                                  slots=dput(slots, dev), n_sel=1)
    else:
        (q.qgemv_rows_mx_swiglu if pair else q.qgemv_rows_mx)(*ws, 0, n, x, y[:, :n])
    got = host(y)
    assert np.isnan(got[:, n:]).all()
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        r = [mxref.product(xv[lo:hi], mxref.values(b[i * n:(i + 1) * n], k), kind) for b in wbs]
        ref, bound = mxref.swiglu(*r[0], *r[1]) if pair else r[0]
        ref = past_range(ref)
        near(got[lo:hi, :n], ref, bound, out, f"expert {i}")


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("tok,n,k", [(1, 40, 64), (4, 2, 160), (5, 300, 2880), (40, 1030, 416), (300, 523, 224),
                                     (2049, 1030, 224)])
def test_largest_scales(dev, kind, pair, tok, n, k):
    check_huge(dev, kind, pair, tok, n, k, "bf16" if tok == 300 else "f32")


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "mxfp4"])
@pytest.mark.parametrize("tok,n,k,n_expert", [(9, 40, 160, 3), (700, 523, 224, 3)])
def test_largest_scales_of_experts(dev, kind, pair, tok, n, k, n_expert):
    check_huge(dev, kind, pair, tok, n, k, n_expert=n_expert)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tok", [3, 700])
def test_largest_scales_beside_others(dev, kind, tok):
    """Rows of finite weights keep their bits where another row is summed in 64 bits, and so do infinities and NaN
    that x or a scale of 255 brings."""
    rng = np.random.default_rng(tok)
    n, k = 530, 224
    wb = mxref.random_blocks(rng, n, k, 115, 121)
    wb.reshape(n, -1, 17)[5, 2, 0] = 255
    xv = rng.standard_normal((tok, k))
    xv[0, 40], xv[2, 3] = np.inf, np.nan
    x = dput(xv.astype(np.float32), dev, kind)
    ys = []
    for huge in (False, True):
        if huge:
            wb.reshape(n, -1, 17)[3::16, 1, 0] = 254
            wb.reshape(n, -1, 17)[3::16, 1, 1:] = 0x77  # 6 * 2^127
        y = nan_buffer(tok, n, "f32", dev)
        q.qgemv_rows_mx(blocks(wb, k, dev), 0, n, x, y)
        ys.append(host(y))
    rest = np.arange(n) % 16 != 3
    assert np.array_equal(ys[0][:, rest], ys[1][:, rest], equal_nan=True)
    assert np.isnan(ys[1][:, 5]).all() and np.isnan(ys[1][2]).all()
    # 6 * 2^127 times the sum of 32 of x: only that decides, and token 0's infinity
    s = host(x)[:, 32:64].sum(1)
    sure = (np.abs(s) > 1.0) & (np.arange(tok) != 2)
    want = np.broadcast_to(np.sign(s[sure])[:, None] * np.inf, (sure.sum(), len(range(3, n, 16))))
    assert sure.sum() >= 1 and np.array_equal(ys[1][sure][:, 3::16], want)


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mxfp4"])
@pytest.mark.parametrize("large_x", [False, True])
@pytest.mark.parametrize("tok,n,k", [(3, 40, 160), (300, 523, 224)])
def test_opposite_scales(dev, kind, pair, large_x, tok, n, k):
    """The scales' ends against each other: weights of scales 0 to 4 (subnormal in fp32 among them) times x about 2^125,
    and weights of scales 250 to 252 times x about 2^-125; every product is an ordinary number."""
    rng = np.random.default_rng(tok + large_x)
    ws = [mxref.random_blocks(rng, n, k, *((0, 5) if large_x else (250, 253))) for _ in range(1 + pair)]
    if kind == "mxfp4":
        b = mxref.random_blocks(rng, tok, k, *((249, 253) if large_x else (0, 5)))
        x, xv = blocks(b, k, dev), mxref.values(b, k)
    else:
        x = rng.uniform(0.5, 1.0, (tok, k)) * rng.choice([-1, 1], (tok, k)) * 2.0 ** (125 if large_x else -125)
        x, xv = as_given(x, kind, dev)
    y = nan_buffer(tok, n, "f32", dev)
    (q.qgemv_rows_mx_swiglu if pair else q.qgemv_rows_mx)(*[blocks(w, k, dev) for w in ws], 0, n, x, y)
    r = [mxref.product(xv, mxref.values(w, k), kind) for w in ws]
    ref, bound = mxref.swiglu(*r[0], *r[1]) if pair else r[0]
    if kind == "f32" and not large_x:
        # x about 2^-125 has bits down to 2^-149; those below 2^-133 are cut off, of each value less than 2^-133
        cut = [2.0 ** -133 * np.abs(mxref.values(w, k)).sum(1)[None] for w in ws]
        bound = bound + (1.1 * cut[0] * np.abs(r[1][0]) + np.abs(r[0][0]) * cut[1] + cut[0] * cut[1] if pair else cut[0])
    near(host(y), ref, bound, "f32")
