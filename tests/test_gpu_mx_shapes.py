"""Every shape of the MXFP4 products (include/qgemv_mx.h) over several stages and
a partial last one, dense and for experts (mx_shapes.py): random operands within
the bounds of mxref.py, exact products bit for bit, infinities and NaN in their
places alone, and the largest scales."""
from __future__ import annotations

import numpy as np
import pytest

import mxref
import quantized_gemv_gguf_amd as q
from mx_shapes import CASES
from test_gpu_mx import T

pytestmark = pytest.mark.gpu

ids = [f"{x}-{'pair' if pair else 'single'}-{shape}-{'experts' if e else 'dense'}" for x, pair, shape, _, _, _, e in CASES]
every_shape = pytest.mark.parametrize("x,pair,shape,places,n,nb,n_expert", CASES, ids=ids)


def values(b):
    """float64 values (rows, k) of blocks (rows, k / 32, 17) on the device."""
    import torch
    c = b[..., 1:].int()
    c = torch.cat([c & 15, c >> 4], -1)
    grid = torch.tensor(mxref.GRID, device=b.device)
    v = torch.where(c >= 8, -1.0, 1.0) * grid[c & 7]
    e = b[..., :1].long()
    scale = torch.where(e == 255, torch.nan, ((e + 896) << 52).view(torch.float64))  # 2^(e - 127)
    return (v * scale).flatten(1)


class Product:
    """One case: operands on the device, their 64-bit values, and the call."""

    def __init__(self, dev, x, pair, places, n, nb, n_expert, seed):
        import torch
        self.x, self.pair, self.n, self.k, self.e = x, pair, n, 32 * nb, max(n_expert, 1)
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self.dev = dev
        rng = np.random.default_rng(seed)
        self.experts = n_expert > 0
        # of experts: sorted places, two behind the last, one expert without any; tokens by slots, two choices each
        self.tokens = (places + 1) // 2 if self.experts else places
        self.places = places
        cuts = [0] + sorted(rng.integers(0, places - 1, self.e - 1)) + [places - 2] if self.experts else [0, places]
        if self.experts:
            cuts[2] = cuts[1]
        self.offsets = [int(c) for c in cuts]
        self.slots = torch.randint(0, 2 * self.tokens, (places,), generator=self.gen, device=dev, dtype=torch.int32)
        self.slots[:3] = torch.tensor([0, 2, 4], dtype=torch.int32, device=dev)  # (the special values' tokens)
        self.w = [self.blocks(self.e * n, 115, 121) for _ in range(1 + pair)]

    def blocks(self, rows, lo, hi):
        import torch
        b = torch.randint(0, 256, (rows, self.k // 32, 17), generator=self.gen, device=self.dev, dtype=torch.uint8)
        b[..., 0] = torch.randint(lo, hi, b.shape[:2], generator=self.gen, device=self.dev).to(torch.uint8)
        return b

    def normal(self):
        import torch
        return torch.randn(self.tokens, self.k, generator=self.gen, device=self.dev)

    def given(self, v):
        """`v` as the call takes it, and its values: floats, or blocks that were quantised on the host's terms."""
        if self.x == "mxfp4":
            return q.Matrix(v, q.MXFP4, v.shape[0], self.k), values(v)
        t = v.to(T(self.x))
        return t, t.double()

    def call(self, x, out="f32"):
        import torch
        y = torch.full((self.places, self.n + 3), float("nan"), dtype=T(out), device=self.dev)
        ws = [q.Matrix(w, q.MXFP4, self.e * self.n, self.k) for w in self.w]
        if self.experts:
            (q.qgemv_expert_mx_swiglu if self.pair else q.qgemv_expert_mx)(
                *ws, self.e, x, torch.tensor(self.offsets, dtype=torch.int32, device=self.dev), y[:, :self.n],
                slots=self.slots, n_sel=2)
        else:
            (q.qgemv_rows_mx_swiglu if self.pair else q.qgemv_rows_mx)(*ws, 0, self.n, x, y[:, :self.n])
        assert torch.isnan(y[self.offsets[-1]:]).all() and torch.isnan(y[:, self.n:]).all(), "wrote beyond the places"
        return y[:, :self.n].double()

    def parts(self, xv):
        """(places, values of their x, values of the expert's weights) of each expert that has places."""
        at = (self.slots // 2).long() if self.experts else None
        for i in range(self.e):
            lo, hi = self.offsets[i], self.offsets[i + 1]
            if lo < hi:
                xs = xv[at[lo:hi]] if self.experts else xv
                yield slice(lo, hi), xs, [values(w[i * self.n:(i + 1) * self.n]) for w in self.w]

    def reference(self, xs, ws):
        """(product or SwiGLU pair in 64 bits, its bound): the formulas of mxref.py on the device."""
        import torch
        step = 4 * np.ceil(mxref.STEPS[self.x] * self.k) * 2.0 ** -23
        r = [(xs @ w.T, step * (xs.abs() @ w.abs().T)) for w in ws]
        if not self.pair:
            return r[0]
        (g, dg), (u, du) = r
        s = g / (1 + torch.exp(-g))
        h = s * u
        return h, 1.1 * dg * (u.abs() + du) + s.abs() * du + (g.abs() + 8) * 2.0 ** -24 * h.abs()


def check(got, ref, bound, out, what):
    """As mxref.near, on the device."""
    import torch
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities"
    fine = torch.isfinite(ref)
    b = bound[fine]
    allowed = b + mxref.HALF[out] * (ref[fine].abs() + b) + mxref.TINY[out]
    err = (got[fine] - ref[fine]).abs()
    assert bool((err <= allowed).all()), f"{what}: worst {float((err / allowed).max()):.3g} times the bound"


@every_shape
def test_random(dev, x, pair, shape, places, n, nb, n_expert):
    p = Product(dev, x, pair, places, n, nb, n_expert, 1)
    out = ["f32", "bf16", "f16"][(shape + pair) % 3]
    xg, xv = p.given(p.blocks(p.tokens, 122, 129) if x == "mxfp4" else p.normal())
    got = p.call(xg, out)
    for at, xs, ws in p.parts(xv):
        check(got[at], *p.reference(xs, ws), out, f"places {at}")


@every_shape
def test_exact(dev, x, pair, shape, places, n, nb, n_expert):
    """Each row of W picks one value of x, which comes back with all its bits: 24 of fp32 x, whose three terms lie in
    places of their own.  Of a pair, silu(64) = 64 and silu(g) = g for g of 32 and more in fp32 (exp(-32) is far below
    half a step of 1), so that with 64 or 1 on the other side the product has the picked bits too."""
    import torch
    p = Product(dev, x, pair, places, n, nb, n_expert, 2)
    k, rows = p.k, p.e * n
    if x == "mxfp4":
        v = p.blocks(p.tokens, 131, 134)
        v[..., 1:] = (v[..., 1:] & 0x77) | 0x44   # 2 .. 6 of scales 2^4 to 2^6: 32 and more
        v[:, 0, 1:] |= 0x66                       # (the first block: 4 and 6)
        v[:, 0, 0] = 131
        v[:, 0, 1:3] = 0x66                       # x[0] = x[1] = 64 there
    else:
        v = 64 * (1 + torch.rand(p.tokens, k, generator=p.gen, device=dev))
        v[:, :2] = 64.0
    xg, xv = p.given(v)
    pick = torch.randint(2, k, (rows,), generator=p.gen, device=dev)
    one = torch.arange(rows, device=dev)

    def picking(column, scale):
        b = torch.zeros(rows, k // 32, 17, dtype=torch.uint8, device=dev)
        b[..., 0] = 127
        j = column % 32
        b[one, column // 32, 0] = scale
        b[one, column // 32, 1 + j % 16] = (2 << (4 * (j // 16))).to(torch.uint8)  # code 2: 1.0
        return b

    p.w[0] = picking(pick, 127)
    if pair:
        # even rows: gate picks the value, up 64 * 2^-6; odd rows: gate 64, up the value
        even = one % 2 == 0
        p.w[0][~even] = picking(torch.ones_like(pick), 127)[~even]
        p.w.append(picking(pick, 127))
        p.w[1] = torch.where(even[:, None, None], picking(torch.zeros_like(pick), 121), p.w.pop())
    got = p.call(xg)
    at = (p.slots // 2).long() if p.experts else torch.arange(places, device=dev)
    for i in range(p.e):
        lo, hi = p.offsets[i], p.offsets[i + 1]
        rows_i = slice(i * n, (i + 1) * n)
        want = xv[at[lo:hi]][:, pick[rows_i]]
        if pair:
            want = want * torch.where(even[rows_i], 1.0, 64.0)
        assert torch.equal(got[lo:hi], want), f"expert {i}"


@every_shape
def test_special_values(dev, x, pair, shape, places, n, nb, n_expert):
    """Token 0 holds an infinity (4-bit: a block of NaN), token 1 a NaN, in the last stage; row 3 of W (of the up matrix
    row 7) a block of scale 255, row 9 subnormal weights, row 11 zeros of both signs: nothing else is touched."""
    import torch
    p = Product(dev, x, pair, places, n, nb, n_expert, 3)
    at_inf, at_nan = p.k - 3, p.k - 40
    for i in range(p.e):
        p.w[0][i * n + 3, nb // 2, 0] = 255
        if pair:
            p.w[1][i * n + 7, nb - 1, 0] = 255
        p.w[0][i * n + 9, :, 0] = 0
        p.w[0][i * n + 11, :, 1:] = torch.randint(0, 2, (nb, 16), generator=p.gen, device=dev, dtype=torch.uint8) * 0x88
    if x == "mxfp4":
        v = p.blocks(p.tokens, 122, 129)
        v[0, at_inf // 32, 0] = v[1, at_nan // 32, 0] = 255
    else:
        v = p.normal()
        v[0, at_inf], v[1, at_nan] = float("inf"), float("nan")
    xg, xv = p.given(v)
    bad = torch.zeros(p.tokens, dtype=torch.bool, device=dev)
    bad[1] = True
    bad[0] = x == "mxfp4"
    infinite = torch.isinf(xv).any(1)
    xv = torch.nan_to_num(xv, nan=0.0, posinf=0.0)
    got = p.call(xg)
    token = (p.slots // 2).long() if p.experts else torch.arange(places, device=dev)
    for at, xs, ws in p.parts(xv):
        hit = [torch.isnan(w).any(1) for w in ws]
        ws = [torch.nan_to_num(w, nan=0.0) for w in ws]
        ref, bound = p.reference(xs, ws)
        # the infinity times its column: of a pair silu(inf) inf; silu(-inf) is -inf * 0
        sign = [torch.sign(w[:, at_inf]) for w in ws]
        nan = torch.tensor(float("nan"), device=dev, dtype=torch.float64)
        if pair:
            # (a zero weight there makes g or u NaN)
            row = torch.where((sign[0] > 0) & (sign[1] != 0), sign[1] * torch.inf, nan)
        else:
            row = torch.where(sign[0] != 0, sign[0] * torch.inf, nan)
        ref = torch.where(infinite[token[at], None], row[None], ref)
        wrong = bad[token[at], None] | torch.stack(hit).any(0)[None]
        check(got[at], torch.where(wrong, nan, ref), bound, "f32", f"places {at}")


@every_shape
def test_largest_scales(dev, x, pair, shape, places, n, nb, n_expert):
    """Scales 250 to 254 in a block of every seventh row, whose products with small x are ordinary and with zeros
    zero."""
    import torch
    p = Product(dev, x, pair, places, n, nb, n_expert, 4)
    for i, w in enumerate(p.w):
        r = torch.arange(3 * i, p.e * n, 7, device=dev)
        w[r, 1 + r % (nb - 1), 0] = (250 + r // 7 % 5).to(torch.uint8)
    tokens = torch.arange(p.tokens, device=dev)
    if x == "mxfp4":
        v = p.blocks(p.tokens, 122, 129)
        v[..., 0] -= torch.where(tokens % 3 == 0, 0, torch.where(tokens % 3 == 1, 100, 12))[:, None].to(torch.uint8)
        v[tokens % 3 == 0, 1:, 1:] = 0
    else:
        v = p.normal()
        v *= torch.where(tokens % 3 == 1, 2.0 ** (-14 if x == "f16" else -100), 2.0 ** -12)[:, None]
        v[tokens % 3 == 0, 32:] = 0.0
    xg, xv = p.given(v)
    got = p.call(xg)
    for at, xs, ws in p.parts(xv):
        ref, bound = p.reference(xs, ws)
        check(got[at], ref, bound, "f32", f"places {at}")
