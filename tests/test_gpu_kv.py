"""GPU parity of the paged cache's operators (include/qgemv_kv.h) against plain 64-bit forms (kvref.py, where the bounds
are derived): rotary positions and their gradient, writes into the cache, attention, the pages' bookkeeping, and the
calls together as a decoder uses them."""
from __future__ import annotations

import math
import random

import pytest
import torch

import kvref
import quantized_gemv_gguf_amd as q
from kvref import TYPES

pytestmark = pytest.mark.gpu


def within(got, ref, tol, what):
    """Every value within its bound; the same values are NaN and infinite."""
    got, ref = got.cpu().double(), ref.double()
    assert got.shape == ref.shape
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), what
    over = ((got - ref).abs() / tol.clamp(min=1e-300))[fine]
    assert not over.numel() or float(over.max()) <= 1.0, f"{what}: {float(over.max()):.3g} times the bound"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(x, dev, pad=0, order=None):
    """x on the device: its axes in memory in `order`, the last one's rows `pad` values longer."""
    order = order or list(range(x.dim()))
    y = torch.full((*[x.shape[i] for i in order[:-1]], x.shape[-1] + pad), float("nan"), dtype=x.dtype, device=dev)
    y = y[..., :x.shape[-1]].permute([order.index(i) for i in range(x.dim())])
    y.copy_(x)
    return y


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def rope_of(rot, dev, interleaved=False, scaling=q.ROPE_NONE, mscale=None):
    f, m = q.qgemv_rope_freqs(rot, 10000.0, scaling, 8.0)
    return q.Rope(torch.tensor(f, dtype=torch.float64, device=dev), interleaved, m if mscale is None else mscale)


# --- rotary positions ----------------------------------------------------------------

ROPES = [(1, 64, 96, 24), (1, 1, 2, 2), (7, 3, 64, 64), (130, 2, 80, 10), (33, 5, 128, 56), (300, 8, 128, 128),
         (5, 1, 65, 2), (2000, 2, 256, 256), (3, 1, 1100, 1024), (65, 7, 33, 16), (20000, 1, 8, 4)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("x,y", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n,h,d,rot", ROPES)
def test_rope(dev, n, h, d, rot, x, y, interleaved):
    g = gen(n * 7 + d)
    a = (torch.randn(n, h, d, generator=g) * 2).to(TYPES[x])
    pos = torch.randint(0, 1 << 20, (n,), generator=g).int()
    pos[0] = 0
    if n > 2:
        pos[1], pos[2] = 2 ** 31 - 1, -5
    r = rope_of(rot, dev, interleaved, q.ROPE_YARN)
    for inverse in (False, True):
        out = strided(torch.full((n, h, d), 7.0, dtype=TYPES[y]), dev, 3)
        q.qgemv_rope(strided(a, dev, 5), pos.to(dev), r, out, inverse=inverse)
        ref, big = kvref.turned(a, pos, r.freqs.cpu(), interleaved, r.mscale, inverse)
        tol = kvref.turn_bound(ref, big, pos, r.freqs.cpu(), TYPES[y])
        within(out, ref, tol, f"rope {inverse}")
        if x == y:
            assert torch.equal(out[..., rot:].cpu(), a[..., rot:])
        base = out.as_strided((n * h, d + 3), (d + 3, 1))
        assert torch.isnan(base[:-1, d:]).all(), "wrote between the heads"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rope_in_place_and_by_heads(dev, kind, interleaved):
    """In place; and tokens within heads in memory; have the bits of the other ways."""
    a = torch.randn(37, 6, 96, generator=gen(3)).to(TYPES[kind]).to(dev)
    pos = torch.arange(100, 137, dtype=torch.int32, device=dev)
    r = rope_of(24, dev, interleaved)
    out = torch.empty_like(a)
    q.qgemv_rope(a, pos, r, out)
    b = strided(a, dev, 8, [1, 0, 2])
    c = strided(torch.zeros_like(a), dev, 0, [1, 0, 2])
    q.qgemv_rope(b, pos, r, c)
    assert torch.equal(c, out)
    q.qgemv_rope(b, pos, r, b)
    assert torch.equal(b, out)


def test_rope_gradient(dev):
    """The inverse is the gradient: by the formula's adjoint, and by differences."""
    n, h, d, rot = 5, 2, 32, 20
    g = gen(9)
    x, dy = torch.randn(n, h, d, generator=g), torch.randn(n, h, d, generator=g)
    pos = torch.randint(0, 5000, (n,), generator=g).int().to(dev)
    for interleaved in (False, True):
        r = rope_of(rot, dev, interleaved, mscale=1.25)
        y, dx = torch.empty(n, h, d, device=dev), torch.empty(n, h, d, device=dev)
        q.qgemv_rope(x.to(dev), pos, r, y)
        q.qgemv_rope(dy.to(dev), pos, r, dx, inverse=True)
        # <dy, R x> = <R^T dy, x>: each side a sum of n h d products whose factors round by 10 half-steps
        left, right = (y.cpu().double() * dy).sum(), (dx.cpu().double() * x).sum()
        assert abs(left - right) <= 1.25 * 2 * (x.abs() * dy.abs().amax()).double().sum() * 10 * 2.0 ** -24
        # the turn is linear, so a step of 1 is its derivative
        e = torch.zeros(n, h, d)
        e[2, 1, 3] = 1.0
        z = torch.empty(n, h, d, device=dev)
        q.qgemv_rope(e.to(dev), pos, r, z)
        assert abs(float((z.cpu().double() * dy).sum()) - float(dx[2, 1, 3])) <= 4 * 1.25 * 10 * 2.0 ** -24 * float(dy.abs().max())


# --- a batch over a paged cache --------------------------------------------------------

ORDERS = [[0, 1, 2, 3, 4], [0, 1, 3, 2, 4], [1, 0, 2, 3, 4], [3, 2, 1, 0, 4]]


class Batch:
    """Sequences with `new` new tokens of `lens` positions each, pages without order, unused memory full of NaN."""

    def __init__(self, dev, lens, new, kv, dim, kind="f16", size=16, layers=2, order=0, pad=0, room=2, seed=1, spare=3):
        g = gen(seed)
        self.dev, self.size, self.lens, self.new = dev, size, lens, new
        each = [max(0, -(-n // size)) for n in lens]
        total = sum(each)
        perm = torch.randperm(total + spare, generator=g).tolist()
        self.tables = torch.full((len(lens), max(each + [0]) + room), -1, dtype=torch.int32)
        shape = (layers, total + spare, kv, size, dim)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=TYPES[kind]) for _ in range(2))
        for s, n in enumerate(each):
            mine = [perm.pop() for _ in range(n)]
            self.tables[s, :n] = torch.tensor(mine, dtype=torch.int32)
            for i, p in enumerate(mine):
                m = min(size, lens[s] - i * size)
                for t in (self.k, self.v):
                    t[:, p, :, :m] = torch.randn(layers, kv, m, dim, generator=g).to(t.dtype)
        self.starts = [0]
        for n in new:
            self.starts.append(self.starts[-1] + n)
        self.rows = self.starts[-1]
        self.cache = q.KvCache(strided(self.k, dev, pad, ORDERS[order]), strided(self.v, dev, pad, ORDERS[order]))
        self.reload()

    def reload(self):
        self.seqs = q.KvSeqs(ints(self.starts, self.dev), ints(self.lens, self.dev), self.tables.to(self.dev))
        self.cache.k.copy_(self.k)
        self.cache.v.copy_(self.v)


def attend(b, x, out_kind, layer=1, behind=2, pad=0, stream=None, **kw):
    """(out, lse) of the call, on rows and a workspace that hold NaN before; `behind` rows belong to no sequence."""
    rows, heads, dim = x.shape
    dev = b.dev
    xd = strided(torch.cat([x, torch.full((behind, heads, dim), float("nan"), dtype=x.dtype)]), dev, pad)
    out = strided(torch.full((rows + behind, heads, dim), 7.0, dtype=TYPES[out_kind]), dev, pad)
    lse = torch.full((rows + behind, heads), 7.0, device=dev)
    work = torch.full((q.qgemv_kv_attend_bytes(xd, b.seqs, b.cache) // 4,), float("nan"), device=dev)
    if kw.get("sinks") is not None:
        kw["sinks"] = kw["sinks"].to(dev)
    q.qgemv_kv_attend(xd, b.seqs, b.cache, layer, out, lse=lse, work=work, stream=stream, **kw)
    assert (out[rows:] == 7.0).all() and (lse[rows:] == 7.0).all(), "rows of no sequence were written"
    return out[:rows], lse[:rows]


def check_attend(b, x, out_kind, layer=1, scale=0.3, what="", **kw):
    r = kvref.attended(x, b.starts, b.lens, b.tables, b.k, b.v, layer, scale,
                       **{n: kw[n] for n in ("causal", "window", "sinks") if n in kw})
    assert r["mine"].all()
    out, lse = attend(b, x, out_kind, layer, scale=scale, **kw)
    wide = not (x.dtype == b.k.dtype == TYPES[out_kind])
    tol, tol_lse = kvref.bounds(r, x.shape[2], b.k.dtype, TYPES[out_kind], wide)
    within(out, r["out"], tol, f"{what} out")
    within(lse, r["lse"], tol_lse, f"{what} lse")
    return out, lse


def queries(b, heads, dim, kind, seed=5, size=1.5):
    return (torch.randn(b.rows, heads, dim, generator=gen(seed)) * size).to(TYPES[kind])


DIMS = [32, 64, 96, 128, 160, 192, 224, 256]
KINDS = [("f16", "f16", "f16"), ("bf16", "bf16", "bf16"), ("f32", "f16", "f32"), ("f32", "bf16", "f32"),
         ("f16", "bf16", "f16"), ("bf16", "f16", "f32"), ("bf16", "bf16", "f32")]


@pytest.mark.parametrize("x,c,y", KINDS)
@pytest.mark.parametrize("dim", DIMS)
def test_attend_heads_and_types(dev, dim, x, c, y):
    """Tokens and short chunks of sequences of many lengths, queries shared by heads."""
    b = Batch(dev, [1, 37, 300, 128, 2], [1, 1, 5, 2, 2], 2, dim, c, seed=dim)
    check_attend(b, queries(b, 6, dim, x), y)


@pytest.mark.parametrize("x,c,y", KINDS)
@pytest.mark.parametrize("dim", DIMS)
def test_attend_prompts_heads_and_types(dev, dim, x, c, y):
    """Chunks of prompts, partial tiles of rows and keys among them."""
    b = Batch(dev, [150, 61, 200], [75, 61, 1], 1, dim, c, seed=dim)
    check_attend(b, queries(b, 2, dim, x), y)
    check_attend(b, queries(b, 2, dim, x), y, window=50)


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513]


@pytest.mark.parametrize("size", [1, 2, 4, 16, 128])
@pytest.mark.parametrize("group", [1, 4])
def test_attend_lengths(dev, group, size):
    """One token of each length about the pieces of the keys, any page size."""
    b = Batch(dev, LENGTHS, [1] * len(LENGTHS), 1, 64, "bf16", size, seed=size)
    check_attend(b, queries(b, group, 64, "bf16"), "bf16")


CHUNKS = [([40], [40]), ([64], [33]), ([129, 5], [129, 1]), ([300, 40, 0, 7, 90], [17, 0, 0, 7, 64]),
          ([10, 3], [16, 7]), ([0, 5], [3, 5]), ([600], [200]), ([257], [256])]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 20, 130])
@pytest.mark.parametrize("i", range(len(CHUNKS)))
def test_attend_chunks(dev, i, window, causal):
    """Ragged chunks, with no new tokens, no positions, and more new tokens than positions (rows that see nothing)."""
    lens, new = CHUNKS[i]
    b = Batch(dev, lens, new, 2, 64, "f16", 16, seed=i)
    sinks = torch.randn(6, generator=gen(i))
    out, lse = check_attend(b, queries(b, 6, 64, "f16"), "f16", causal=causal, window=window)
    if causal:
        for s, (n, m) in enumerate(zip(lens, new)):
            for t in range(max(0, m - n)):
                assert (out[b.starts[s] + t] == 0).all() and (lse[b.starts[s] + t] == -math.inf).all()
    check_attend(b, queries(b, 6, 64, "f16"), "f16", causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 16, 17, 40])
def test_attend_groups(dev, group):
    b = Batch(dev, [50, 200], [3, 30], 2, 96, "f16", seed=group)
    check_attend(b, queries(b, 2 * group, 96, "f16"), "f16")


@pytest.mark.parametrize("order", range(len(ORDERS)))
@pytest.mark.parametrize("new", [1, 70])
def test_attend_layouts(dev, order, new):
    """Caches whose axes lie in other orders, rows that are slices of longer ones: the same bits."""
    b = Batch(dev, [150, 90], [new, new], 3, 64, "bf16", seed=4)
    x = queries(b, 6, 64, "bf16")
    out, lse = check_attend(b, x, "bf16")
    c = Batch(dev, [150, 90], [new, new], 3, 64, "bf16", seed=4, order=order, pad=8)
    out2, lse2 = attend(c, x, "bf16", pad=3, scale=0.3)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new", [1, 9, 60])
def test_attend_lengths_past_the_table(dev, new, causal):
    """Positions that the table does not hold are masked, and do not move the others; the widest window hides nothing,
    nor does it where rows lie before the sequence's start."""
    b = Batch(dev, [150, 40, 48], [new, new, new], 2, 64, "bf16", 16, seed=9, room=0)
    b.tables = b.tables[:, :5].contiguous()  # 80 positions
    b.lens[1] = 2 ** 31 - 1 if causal else 79
    b.reload()
    x = queries(b, 4, 64, "bf16")
    for window in (0, 2 ** 31 - 1, 100):
        if b.lens[1] > 1000:  # (the plain form's last sequence would see its whole window past the table)
            ref = [min(n, 10 ** 6) for n in b.lens]
        else:
            ref = b.lens
        r = kvref.attended(x, b.starts, ref, b.tables, b.k, b.v, 1, 0.3, causal=causal, window=window)
        out, lse = attend(b, x, "bf16", scale=0.3, causal=causal, window=window)
        tol, tol_lse = kvref.bounds(r, 64, torch.bfloat16, torch.bfloat16, False)
        within(out, r["out"], tol, "out")
        within(lse, r["lse"], tol_lse, "lse")
    c = Batch(dev, [10, 3], [40, 3], 1, 64, "f16", 16, seed=9)
    check_attend(c, queries(c, 2, 64, "f16"), "f16", window=2 ** 31 - 1)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_attend_pages_that_are_not_there(dev, kind, new):
    """Positions of unmapped pages are masked, so are those of ids out of range."""
    b = Batch(dev, [200, 64, 48], [new, new, new], 2, 64, kind, 16, seed=2)
    for s, p, bad in [(0, 0, -1), (0, 3, b.k.shape[1]), (0, 4, 2 ** 31 - 1), (1, 1, -2 ** 31), (2, 0, -7), (2, 1, -7), (2, 2, 999)]:
        b.tables[s, p] = bad
    b.reload()
    out, lse = check_attend(b, queries(b, 4, 64, kind), kind)
    assert (out[-new:] == 0).all() and (lse[-new:] == -math.inf).all()


@pytest.mark.parametrize("new", [1, 30, 70])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_attend_masked_places_do_not_matter(dev, kind, new):
    """Infinities and NaN in keys and values that a row may not see; rows that see them get what IEEE makes of them."""
    b = Batch(dev, [90, 200], [new, new], 1, 64, kind, 16, seed=6)
    x = queries(b, 2, 64, kind)
    for s, n in enumerate(b.lens):
        last = n - 1
        page, slot = int(b.tables[s, last // 16]), last % 16
        b.v[1, page, 0, slot, 3], b.v[1, page, 0, slot, 4], b.v[1, page, 0, slot, 5] = math.inf, -math.inf, math.nan
        if n > 40:  # seen by the later rows of a window only
            page, slot = int(b.tables[s, (n - 40) // 16]), (n - 40) % 16
            b.v[1, page, 0, slot, 3] = -math.inf
            b.v[1, page, 0, slot, 7] = math.inf
    b.reload()
    for window in (0, 30):
        out, _ = check_attend(b, x, kind, window=window)
        assert torch.isfinite(out[:new - 1, :, 8:]).all()
        assert torch.isnan(out[new - 1, :, 5]).all()
    # keys without a size, hidden by the window and by the order
    c = Batch(dev, [90, 200], [new, new], 1, 64, kind, 16, seed=6)
    for s, n in enumerate(c.lens):
        for j in (n - 1, n - 60):
            c.k[1, int(c.tables[s, j // 16]), 0, j % 16] = math.nan
    c.reload()
    out, _ = attend(c, x, kind, window=15, scale=0.3)
    for s, n in enumerate(c.lens):
        for i in range(new):
            pos = n - new + i
            sees = any(pos - 15 < j <= pos for j in (n - 1, n - 60))
            row = out[c.starts[s] + i]
            assert torch.isnan(row).all() if sees else torch.isfinite(row).all()


def test_attend_large_scores(dev):
    """Scores far apart: weights underflow, sums stay; and q of great and small size in an fp16 cache."""
    b = Batch(dev, [300], [4], 1, 64, "f16", seed=8)
    check_attend(b, queries(b, 2, 64, "f16", size=30.0), "f16", scale=1.0)
    for size in (1e-6, 3e5, 1e9):
        x = queries(b, 2, 64, "f32", size=size)
        check_attend(b, x, "f32", scale=0.5 / size, what=f"size {size}")


def test_attend_long(dev):
    """A long context cut into parts: against fp64 on the device."""
    n, heads, kv, dim = 70001, 4, 2, 128
    for kind, y in (("bf16", "bf16"), ("f16", "f32")):
        g = torch.Generator(device=dev).manual_seed(3)
        pages = -(-n // 64)
        k, v = (torch.randn(1, pages, kv, 64, dim, generator=g, device=dev).to(TYPES[kind]) for _ in range(2))
        table = torch.randperm(pages, generator=g, device=dev).int()[None]
        x = torch.randn(3, heads, dim, generator=g, device=dev).to(TYPES[y])
        cache, seqs = q.KvCache(k, v), q.KvSeqs(ints([0, 3], dev), ints([n], dev), table)
        out, lse = torch.zeros_like(x), torch.zeros(3, heads, device=dev)
        work = torch.empty(q.qgemv_kv_attend_bytes(x, seqs, cache), dtype=torch.uint8, device=dev)
        q.qgemv_kv_attend(x, seqs, cache, 0, out, scale=dim ** -0.5, lse=lse, work=work)
        kk, vv = (t[0, table[0].long()].transpose(0, 1).reshape(kv, -1, dim)[:, :n].double() for t in (k, v))
        r = {n_: torch.zeros(3, heads, dim, dtype=torch.float64) for n_ in ("out", "mean", "total")}
        r.update({n_: torch.zeros(3, heads, dtype=torch.float64) for n_ in ("lse", "worst", "count")})
        for i in range(3):
            for h in range(heads):
                m = n - 2 + i
                a = kk[h // 2, :m] @ x[i, h].double() * dim ** -0.5
                w = torch.softmax(a, 0)
                r["out"][i, h], r["mean"][i, h] = (w @ vv[h // 2, :m]).cpu(), (w @ vv[h // 2, :m].abs()).cpu()
                r["lse"][i, h], r["count"][i, h] = torch.logsumexp(a, 0).cpu(), m
                r["worst"][i, h] = (kk[h // 2, :m].abs() @ x[i, h].double().abs()).max().cpu() * dim ** -0.5
                r["total"][i, h] = (vv[h // 2, :m].abs().sum(0) / torch.exp(a - a.max()).sum()).cpu()
        tol, tol_lse = kvref.bounds(r, dim, TYPES[kind], TYPES[y], kind != y)
        within(out, r["out"], tol, "out")
        within(lse, r["lse"], tol_lse, "lse")


@pytest.mark.parametrize("n_seq", [63, 64, 65, 200, 1000])
def test_attend_many_sequences(dev, n_seq):
    """Sequences found over several rounds of a wave, some without rows."""
    r = random.Random(n_seq)
    lens = [r.choice([0, 1, 5, 40, 200]) for _ in range(n_seq)]
    new = [0 if r.random() < 0.2 else 1 if r.random() < 0.8 else 3 for _ in range(n_seq)]
    b = Batch(dev, lens, new, 1, 32, "f16", 16, seed=n_seq)
    check_attend(b, queries(b, 2, 32, "f16"), "f16")


def test_attend_twice_and_on_a_stream(dev):
    """The same bits again, on another stream, and beside another call with a workspace of its own."""
    b = Batch(dev, [3000, 10, 500], [1, 1, 1], 2, 64, "bf16", seed=11)
    x = queries(b, 8, 64, "bf16")
    first = attend(b, x, "bf16", scale=0.2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = attend(b, x, "bf16", scale=0.2)
    third = attend(b, x, "bf16", scale=0.2)
    torch.cuda.synchronize()
    for a, c, d in zip(first, second, third):
        assert torch.equal(a, c) and torch.equal(a, d)


# --- writes into the cache ---------------------------------------------------------------

@pytest.mark.parametrize("x,c", [("f32", "f16"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "bf16")])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (24, False), (24, True), (96, False), (10, False)])
def test_append(dev, x, c, rot, interleaved):
    """Keys turned and values as they are into their slots, nothing else touched; queries turned; rows of no sequence,
    without a page or before the sequence's start stay away."""
    b = Batch(dev, [20, 3, 70, 0, 40], [5, 3, 33, 2, 0], 2, 96, c, 16, seed=rot)
    b.tables[2, 3] = 9999
    b.tables[0, 1] = -1
    b.reload()
    n, behind = b.rows, 3
    g = gen(1)
    row = torch.randn(n + behind, 10 * 96, generator=g).to(TYPES[x]).to(dev)
    xq, xk, xv = (t.unflatten(1, (-1, 96)) for t in row.split([6 * 96, 2 * 96, 2 * 96], 1))
    r = rope_of(rot, dev, interleaved) if rot else None
    out = torch.full((n + behind, 6, 96), 7.0, dtype=TYPES[x], device=dev)
    k0, v0 = b.cache.k.clone(), b.cache.v.clone()
    q.qgemv_kv_append(xk, xv, b.seqs, b.cache, 1, rope=r, **(dict(q=xq, q_out=out) if rot else {}))
    pos = torch.zeros(n, dtype=torch.int32)
    for s in range(5):
        for i in range(b.new[s]):
            pos[b.starts[s] + i] = b.lens[s] - b.new[s] + i
    freqs = r.freqs.cpu() if rot else torch.zeros(0, dtype=torch.float64)
    m = r.mscale if rot else 1.0
    want_k, want_v = k0.cpu().double(), v0.cpu().double()
    tol_k = torch.zeros_like(want_k)
    turned, big = kvref.turned(xk[:n].cpu(), pos, freqs, interleaved, m)
    if rot:
        bound = kvref.turn_bound(turned, big, pos, freqs, TYPES[c])
    else:
        bound = turned.abs() * kvref.EPS[TYPES[c]] + kvref.TINY[TYPES[c]]
    for s in range(5):
        for i in range(b.new[s]):
            t = b.starts[s] + i
            p = int(pos[t])
            page = int(b.tables[s, p // 16]) if p >= 0 else -1
            if 0 <= page < k0.shape[1]:
                want_k[1, page, :, p % 16], tol_k[1, page, :, p % 16] = turned[t], bound[t]
                want_v[1, page, :, p % 16] = xv[t].cpu().to(TYPES[c]).double()
    within(b.cache.k, want_k, tol_k, "keys")
    within(b.cache.v, want_v, torch.zeros_like(want_v), "values")
    if rot:
        ref, big = kvref.turned(xq[:n].cpu(), pos, freqs, interleaved, m)
        within(out[:n], ref, kvref.turn_bound(ref, big, pos, freqs, TYPES[x]), "queries")
        assert (out[n:] == 7.0).all()
        # positions of their own, for the turn alone; in place
        given = torch.arange(1000, 1000 + n + behind, dtype=torch.int32, device=dev)
        want = torch.empty_like(out)
        q.qgemv_rope(xq, given, r, want)
        q.qgemv_kv_append(xk, xv, b.seqs, b.cache, 0, rope=r, pos=given, q=xq, q_out=xq)
        assert torch.equal(xq[:n], want[:n])
        kk = torch.empty(n + behind, 2, 96, dtype=TYPES[c], device=dev)
        q.qgemv_rope(xk, given, r, kk)
        page = int(b.tables[1, 0])
        assert torch.equal(b.cache.k[0, page, :, :3].transpose(0, 1), kk[b.starts[1]:b.starts[2]])


@pytest.mark.parametrize("n_seq", [1, 64, 65, 700, 4096])
def test_append_finds_its_sequence(dev, n_seq):
    r = random.Random(n_seq)
    new = [r.choice([0, 1, 1, 2]) for _ in range(n_seq)]
    new[-1] = 1
    b = Batch(dev, [n + r.randint(0, 9) for n in new], new, 1, 32, "f16", 8, layers=1, seed=1)
    x = torch.arange(b.rows * 32, dtype=torch.float32).view(-1, 1, 32).remainder(2047).to(dev)
    q.qgemv_kv_append(x, -x, b.seqs, b.cache, 0)
    for s in r.sample(range(n_seq), min(n_seq, 50)):
        for i in range(new[s]):
            p = b.lens[s] - new[s] + i
            page = int(b.tables[s, p // 8])
            assert torch.equal(b.cache.k[0, page, 0, p % 8].float(), x[b.starts[s] + i, 0])
            assert torch.equal(b.cache.v[0, page, 0, p % 8].float(), -x[b.starts[s] + i, 0])


# --- the pages -------------------------------------------------------------------------

class DevicePool:
    """The pool on the device beside kvref.Pool; every page's content is its first number."""

    def __init__(self, dev, n_seq, max_pages, n_pages, size, layers=2, heads=1, dim=32, order=0, pad=0):
        self.ref = kvref.Pool(n_seq, max_pages, n_pages, size)
        full = lambda shape, v: torch.full(shape, v, dtype=torch.int32, device=dev)  # noqa: E731
        work = torch.empty(q.qgemv_kv_pool_bytes(n_seq, max_pages, n_pages), dtype=torch.uint8, device=dev).fill_(0xA5)
        self.pool = q.KvPool(full((n_seq, max_pages), -1), full((n_seq,), 0), full((n_pages,), 0),
                             full(((n_pages + 31) // 32,), 0), size, work)
        first = torch.arange(n_pages).view(1, -1, 1, 1, 1).expand(layers, n_pages, heads, size, dim)
        low = (first % 256 + torch.arange(layers).view(-1, 1, 1, 1, 1)).half()
        high = (first // 256 + torch.arange(dim).view(1, 1, 1, 1, -1) + 100 * torch.arange(heads).view(1, 1, -1, 1, 1)
                + 500 * torch.arange(layers).view(-1, 1, 1, 1, 1)).half()
        self.k0, self.v0 = low, high
        self.cache = q.KvCache(strided(low, dev, pad, ORDERS[order]), strided(high, dev, pad, ORDERS[order]))
        self.dev = dev

    def resize(self, lens):
        self.ref.resize(lens)
        q.qgemv_kv_resize(self.pool, self.cache, ints(lens, self.dev))

    def fork(self, parents):
        self.ref.fork(parents)
        q.qgemv_kv_fork(self.pool, ints(parents, self.dev))

    def compact(self):
        self.ref.compact()
        q.qgemv_kv_compact(self.pool, self.cache)

    def check(self, what=""):
        for got, want, name in zip((self.pool.tables, self.pool.lens, self.pool.refs, self.pool.used), self.ref.arrays(),
                                   ("tables", "lens", "refs", "used")):
            assert torch.equal(got.cpu(), want), f"{what}: {name}"
        at = torch.tensor(self.ref.data)
        assert torch.equal(self.cache.k.cpu(), self.k0[:, at]) and torch.equal(self.cache.v.cpu(), self.v0[:, at]), what


SIZES = [(1, 4, 5, 16), (3, 8, 20, 4), (8, 40, 100, 1), (40, 12, 300, 16), (70, 9, 40, 8), (1100, 5, 2500, 2)]


@pytest.mark.parametrize("i", range(len(SIZES)))
def test_pool_steps(dev, i):
    """Random growth (past the pages there are and past the tables), cuts, forks and compaction, step by step."""
    n, wide, pages, size = SIZES[i]
    p = DevicePool(dev, n, wide, pages, size, order=i % 4, pad=8 * (i % 2))
    r = random.Random(i)
    for step in range(12):
        lens = []
        for s in range(n):
            now = p.ref.lens[s]
            lens.append(r.choice([-1, now, now + 1, now + r.randint(0, 2 * size), r.randint(0, wide * size), 0,
                                  max(0, now - r.randint(0, size)), wide * size + (r.random() < 0.2)]))
        p.resize(lens)
        p.check(f"step {step} resize")
        if step % 2:
            p.fork([r.choice([s, s, s, -1, r.randrange(n), r.randrange(n), n, -2]) for s in range(n)])
            p.check(f"step {step} fork")
            grow = [x + 1 for x in p.ref.lens]
            p.resize(grow)
            p.check(f"step {step} grown")
        if step % 3 == 2:
            p.compact()
            p.check(f"step {step} compact")


def test_pool_large(dev):
    """More pages than a round of the workgroup's bits, a prompt longer than its threads."""
    p = DevicePool(dev, 5, 50000, 70001, 2, layers=1)
    p.resize([60001, 2, 30000, 0, 7])
    p.resize([0, -1, -1, 41000, -1])
    p.check("filled")
    p.compact()
    p.check("compact")
    p.fork([2, 3, 2, 3, 1])
    p.resize([x + 3 for x in p.ref.lens])
    p.check("forked")


@pytest.mark.parametrize("heads,size,dim", [(1, 1, 32), (3, 16, 96), (8, 64, 128), (5, 128, 256)])
@pytest.mark.parametrize("order", range(len(ORDERS)))
def test_copy_pages(dev, heads, size, dim, order):
    g = gen(2)
    k, v = (torch.randn(2, 9, heads, size, dim, generator=g).half() for _ in range(2))
    cache = q.KvCache(strided(k, dev, 16, ORDERS[order]), strided(v, dev, 16, ORDERS[order]))
    src, dst = [0, 0, 5, -1, 3, 9, 2], [4, 7, 8, 1, 9, 1, -3]
    q.qgemv_kv_copy(cache, ints(src, dev), ints(dst, dev))
    for a, b in ((0, 4), (0, 7), (5, 8)):
        k[:, b], v[:, b] = k[:, a], v[:, a]
    assert torch.equal(cache.k.cpu(), k) and torch.equal(cache.v.cpu(), v)
    if order == 0:
        base = cache.k.as_strided((2 * 9 * heads * size, dim + 16), (dim + 16, 1))
        assert torch.isnan(base[:-1, dim:]).all(), "wrote between the rows"


# --- the calls together --------------------------------------------------------------------

def decode(dev, steps, kind="bf16", captured=False):
    """A prompt, forked into beams, reordered and grown for some steps: every step's outputs, beside attention without
    pages over each beam's own list of keys and values."""
    n_seq, heads, kv, dim, size, rot, prompt = 4, 4, 2, 64, 4, 16, 21
    g = gen(12)
    ref = kvref.Pool(n_seq, 16, 64, size)
    full = lambda shape, v: torch.full(shape, v, dtype=torch.int32, device=dev)  # noqa: E731
    pool = q.KvPool(full((n_seq, 16), -1), full((n_seq,), 0), full((64,), 0), full((2,), 0), size,
                    torch.empty(q.qgemv_kv_pool_bytes(n_seq, 16, 64), dtype=torch.uint8, device=dev))
    nan = lambda: torch.full((1, 64, kv, size, dim), float("nan"), dtype=TYPES[kind], device=dev)  # noqa: E731
    cache = q.KvCache(nan(), nan())
    r = rope_of(rot, dev)
    made = {}

    def step(rows, starts, xs):
        seqs = q.KvSeqs(starts, pool.lens, pool.tables)
        key = len(rows)
        if key not in made:
            x = torch.empty(key, heads, dim, dtype=TYPES[kind], device=dev)
            made[key] = (x, torch.empty_like(x), torch.empty(q.qgemv_kv_attend_bytes(x, seqs, cache), dtype=torch.uint8, device=dev))
        x, out, work = made[key]
        q.qgemv_kv_append(xs[1], xs[2], seqs, cache, 0, rope=r, q=xs[0], q_out=x)
        q.qgemv_kv_attend(x, seqs, cache, 0, out, scale=dim ** -0.5, work=work)
        return x, out

    own = [[] for _ in range(n_seq)]  # each beam's (key, value) rows
    results = []

    def turned(x, pos):
        y = torch.empty_like(x)
        q.qgemv_rope(x, ints(pos, dev), r, y)
        return y

    def new_rows(n):
        row = torch.randn(n, (heads + 2 * kv) * dim, generator=g).to(TYPES[kind]).to(dev)
        return [t.unflatten(1, (-1, dim)) for t in row.split([heads * dim, kv * dim, kv * dim], 1)]

    def check(x, out, owners):
        for i, (s, upto) in enumerate(owners):
            ks, vs = (torch.stack([o[j] for o in own[s][:upto]]).cpu() for j in (0, 1))
            one = kvref.attended(x[i:i + 1].cpu(), [0, 1], [upto], torch.arange(upto)[None].int(),
                                 ks[None, :, :, None], vs[None, :, :, None], 0, dim ** -0.5)
            tol, _ = kvref.bounds(one, dim, TYPES[kind], TYPES[kind], False)
            within(out[i:i + 1], one["out"], tol, f"beam {s}")

    q.qgemv_kv_resize(pool, cache, ints([prompt, -1, -1, -1], dev))
    xs = new_rows(prompt)
    x, out = step(range(prompt), ints([0, prompt, prompt, prompt, prompt], dev), xs)
    ks = turned(xs[1], list(range(prompt)))
    own[0] = [(ks[i], xs[2][i]) for i in range(prompt)]
    check(x, out, [(0, i + 1) for i in range(prompt)])
    q.qgemv_kv_fork(pool, ints([0, 0, 0, 0], dev))
    own = [list(own[0]) for _ in range(n_seq)]
    pick = random.Random(4)
    starts = ints(range(n_seq + 1), dev)
    grown, parents = full((n_seq,), 0), full((n_seq,), 0)
    inputs = new_rows(n_seq)
    graph = None
    for t in range(steps):
        order = [pick.randrange(n_seq) for _ in range(n_seq)]
        parents.copy_(ints(order, dev))
        grown.fill_(prompt + t + 1)
        for a, b in zip(inputs, new_rows(n_seq)):
            a.copy_(b)

        def body():
            q.qgemv_kv_fork(pool, parents)
            q.qgemv_kv_resize(pool, cache, grown)
            return step(range(n_seq), starts, inputs)

        if not captured:
            x, out = body()
        elif graph is None:
            x, out = body()  # (the first step as it is; the graph takes over its buffers)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                body()
        else:
            graph.replay()
            torch.cuda.synchronize()
        own = [list(own[f]) for f in order]
        ks = turned(inputs[1], [prompt + t] * n_seq)
        for s in range(n_seq):
            own[s].append((ks[s], inputs[2][s].clone()))
        assert pool.lens.tolist() == [prompt + t + 1] * n_seq
        check(x, out, [(s, len(own[s])) for s in range(n_seq)])
        if t == steps // 2:
            q.qgemv_kv_compact(pool, cache)
        results.append(out.clone())
    return results


def test_decode_with_beams(dev):
    """Append, attention, forks, copy on write and compaction together."""
    decode(dev, 9)


def test_decode_captured(dev):
    """The whole step replayed as one graph, with eager work in between: the eager steps' bits."""
    for a, b in zip(decode(dev, 9), decode(dev, 9, captured=True)):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(dev):
    """Pages that lie past 2^32 bytes, and past 2^31 elements, of the cache."""
    pages, kv, size, dim = 70, 1, 16, 64
    base = [torch.zeros(pages << 25, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    k, v = (t.as_strided((1, pages, kv, size, dim), (pages << 25, 1 << 25, size * dim, dim, 1)) for t in base)
    b = Batch(dev, [100, 33], [2, 1], kv, dim, "bf16", size, layers=1, seed=7)
    n = b.k.shape[1]
    at = torch.tensor([0, 69, 68, 33, 64, 65, 66, 67, 1, 2, 3, 4, 5, 6][:n])
    for big, small in ((k, b.k), (v, b.v)):
        big[:, at.to(dev)] = small.to(dev)
    tables = torch.where(b.tables >= 0, at[b.tables.long().clamp(min=0)].int(), -1)
    x = queries(b, 2, dim, "bf16")
    want, _ = attend(b, x, "bf16", 0, scale=0.3)
    b.cache, b.seqs = q.KvCache(k, v), q.KvSeqs(b.seqs.starts, b.seqs.lens, tables.to(dev))
    got, _ = attend(b, x, "bf16", 0, scale=0.3)
    assert torch.equal(got, want)
    q.qgemv_kv_copy(b.cache, ints([69, 1], dev), ints([10, 63], dev))
    assert torch.equal(k[0, 10].nan_to_num(), k[0, 69].nan_to_num()) and torch.equal(v[0, 63].nan_to_num(), v[0, 1].nan_to_num())
    q.qgemv_kv_append(x[:, :1].to(dev), x[:, 1:].to(dev), b.seqs, b.cache, 0)
    page = int(tables[0, 99 // size])
    assert torch.equal(k[0, page, 0, 99 % size].cpu(), x[1, 0]) and torch.equal(v[0, page, 0, 99 % size].cpu(), x[1, 1])


def test_bench_pass_with_attention(dev):
    """The benchmark's pass over a context, eager and replayed: parity of its attention, and room for every token."""
    import json
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for more in ([], ["--eager"]):
        r = subprocess.run([sys.executable, os.path.join(root, "bench.py"), "--workload", "dense20b_context", "--layers", "1",
                            "--context", "37", "--steps", "3", "--warmup", "1", *more], capture_output=True, text=True,
                           timeout=100, cwd=root)
        assert r.returncode == 0, r.stderr[-2000:]
        line = json.loads(r.stdout.strip().splitlines()[-1])
        assert line["parity"]["pass"], line["parity"]


def test_two_graphs_with_workspaces_of_their_own(dev):
    """Two captured calls replayed in turn and at once, with eager work between: every replay has the eager bits."""
    runs = []
    for seed, lens, new, kind in ((1, [3000, 70], [1, 1], "bf16"), (2, [900, 2500], [40, 3], "f16")):
        b = Batch(dev, lens, new, 2, 64, kind, seed=seed)
        x = queries(b, 8, 64, kind).to(dev)
        out, lse = torch.zeros_like(x), torch.zeros(b.rows, 8, device=dev)
        work = torch.empty(q.qgemv_kv_attend_bytes(x, b.seqs, b.cache), dtype=torch.uint8, device=dev)

        def call(b=b, x=x, out=out, lse=lse, work=work):
            q.qgemv_kv_attend(x, b.seqs, b.cache, 1, out, scale=0.2, lse=lse, work=work)

        call()
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, out, lse, want, call))
    side = torch.cuda.Stream()
    for turn in range(4):
        for graph, out, lse, want, call in runs:
            out.fill_(7.0)
            lse.fill_(7.0)
        if turn == 3:
            runs[1][4]()  # eager between
        torch.cuda.synchronize()
        runs[0][0].replay()
        with torch.cuda.stream(side):
            runs[1][0].replay()
        torch.cuda.synchronize()
        for graph, out, lse, want, call in runs:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_append_captured(dev):
    """Lengths that change on the device between replays: each replay stores at its own positions."""
    b = Batch(dev, [40, 9], [2, 1], 2, 64, "f16", seed=3)
    g = gen(5)
    x = torch.randn(3, 2, 64, generator=g).to(dev)
    r = rope_of(64, dev)
    graph = torch.cuda.CUDAGraph()
    q.qgemv_kv_append(x, x, b.seqs, b.cache, 0, rope=r)
    with torch.cuda.graph(graph):
        q.qgemv_kv_append(x, x, b.seqs, b.cache, 0, rope=r)

    def fresh():
        b.cache.k.copy_(b.k)
        b.cache.v.copy_(b.v)

    for lens in ([40, 9], [33, 1], [48, 16], [2, 5]):
        fresh()
        x.copy_(torch.randn(3, 2, 64, generator=g))
        b.seqs.lens.copy_(ints(lens, dev))
        graph.replay()
        torch.cuda.synchronize()
        got = b.cache.k.clone(), b.cache.v.clone()
        fresh()
        q.qgemv_kv_append(x, x, b.seqs, b.cache, 0, rope=r)
        for a, c in zip(got, (b.cache.k, b.cache.v)):
            assert torch.equal(a.nan_to_num(), c.nan_to_num())
        p = lens[1] - 1
        assert torch.equal(b.cache.v[0, int(b.tables[1, p // 16]), :, p % 16], x[2].half())


def test_nothing_to_do(dev):
    """No tokens, no sequences, no pages: outputs stay as they were."""
    b = Batch(dev, [10], [2], 2, 64, "f16")
    x = torch.randn(3, 4, 64, device=dev)
    out = torch.full_like(x, 7.0)
    none = q.KvSeqs(ints([0], dev), ints([], dev), torch.zeros(0, 3, dtype=torch.int32, device=dev))
    q.qgemv_kv_attend(x, none, b.cache, 0, out, scale=1.0)
    q.qgemv_kv_append(x[:, :2], x[:, :2], none, b.cache, 0)
    q.qgemv_kv_attend(x[:0], b.seqs, b.cache, 0, out[:0], scale=1.0, work=torch.empty(1 << 20, dtype=torch.uint8, device=dev))
    q.qgemv_rope(x[:0], ints([], dev), rope_of(64, dev), out[:0])
    q.qgemv_kv_copy(b.cache, ints([], dev), ints([], dev))
    assert (out == 7.0).all() and torch.equal(b.cache.k.nan_to_num().cpu(), b.k.nan_to_num())
    # a table without columns: rows that see nothing
    bare = q.KvSeqs(b.seqs.starts, b.seqs.lens, torch.zeros(1, 0, dtype=torch.int32, device=dev))
    q.qgemv_kv_append(x[:, :2], x[:, :2], bare, b.cache, 0)
    q.qgemv_kv_attend(x, bare, b.cache, 0, out, scale=1.0)
    assert (out[:2] == 0).all() and (out[2:] == 7.0).all()
    assert torch.equal(b.cache.k.nan_to_num().cpu(), b.k.nan_to_num())


def test_attend_keys_about_a_page_end(dev):
    """Parts of the keys that end in a page's last slots, on the cache's last page, few rows and many."""
    for size in (16, 32, 64):
        for n in (size - 1, size, 2 * size - 1, 4 * size - 3, 8 * size - 1):
            for new in (1, min(n, 40)):
                b = Batch(dev, [n], [new], 1, 64, "bf16", size, layers=1, seed=n, spare=0)
                # the pages in order, so that the last one holds the last key
                b.tables = torch.where(b.tables >= 0, torch.arange(b.tables.shape[1], dtype=torch.int32)[None], -1)
                for t in (b.k, b.v):
                    t.copy_(torch.randn(t.shape, generator=gen(n)).to(t.dtype))
                b.reload()
                check_attend(b, queries(b, 2, 64, "bf16"), "bf16", layer=0)
