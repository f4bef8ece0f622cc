"""Plain 64-bit forms of the paged cache's operators (include/qgemv_kv.h), on the CPU, and the bounds of what fp32 sums
and roundings may make of them."""
from __future__ import annotations

import math

import torch

EPS = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the least step
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def turned(x, pos, freqs, interleaved, mscale, inverse=False):
    """(turned heads of x (rows, heads, dim) in 64 bits, the largest magnitudes that met in each value)."""
    half = freqs.numel()
    x = x.double()
    y, big = x.clone(), x.abs()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = pos.double() * freqs[i].double()
        c, s = (torch.cos(t) * mscale)[:, None], (torch.sin(t) * mscale)[:, None]
        s = -s if inverse else s
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        big[..., a] = big[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(mscale)
    return y, big


def turn_bound(ref, big, pos, freqs, kind):
    """Sine and cosine are within 3 half-steps of fp32 of the reduced angle's, that angle within one of fp32 (of at most
    pi / 4) and pos * f of 64 bits (of pos * f); two products and a sum round; the result rounds once."""
    most = float((pos.double().abs().max() * freqs.abs().max()).item()) if pos.numel() else 0.0
    return big * (8 * 2.0 ** -24 + most * 2.0 ** -51) + ref.abs() * EPS[kind] * 1.001 + TINY[kind]


def gathered(cache, layer, table, n, size):
    """(keys or values (heads, n, dim) of the first n positions, which of them are there)."""
    pages = cache.shape[1]
    pos = torch.arange(n)
    page = torch.full((n,), -1, dtype=torch.long)
    inside = pos // size < table.numel()
    page[inside] = table.long()[pos[inside] // size]
    there = (page >= 0) & (page < pages)
    x = cache[layer][page.clamp(0, pages - 1), :, pos % size].double()  # (n, heads, dim)
    return x.transpose(0, 1), there


def attended(q, starts, lens, tables, k, v, layer, scale, causal=True, window=0, sinks=None):
    """(out, lse, tol of out, tol of lse) in 64 bits of rows that belong to a sequence, and which those are.  q in its
    own type, k and v (layers, pages, heads, slots, dim).  The bounds are for weights of relative error `u` and fp32
    sums, see `bounds`."""
    rows, heads, dim = q.shape
    size, kv = k.shape[3], k.shape[2]
    out = torch.zeros(rows, heads, dim, dtype=torch.float64)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64)
    mean = torch.zeros_like(out)        # sum of weights times |v|
    worst = torch.zeros(rows, heads, dtype=torch.float64)  # largest scale * sum |q| |k| of a seen key
    total_v = torch.zeros_like(out)     # sum of |v| over the keys, per unit of the denominator
    count = torch.zeros(rows, heads, dtype=torch.float64)
    mine = torch.zeros(rows, dtype=torch.bool)
    for s in range(len(lens)):
        lo, hi = int(starts[s]), int(starts[s + 1])
        n, length = hi - lo, int(lens[s])
        held = min(length, tables.shape[1] * size)
        if n <= 0:
            continue
        mine[lo:hi] = True
        ks, there = gathered(k, layer, tables[s], held, size)
        vs, _ = gathered(v, layer, tables[s], held, size)
        j = torch.arange(held)
        for i in range(n):
            p = length - n + i
            seen = there.clone()
            if causal:
                seen &= j <= p
            if window:
                seen &= j > p - window
            for h in range(heads):
                kk, vv = ks[h // (heads // kv)][seen], vs[h // (heads // kv)][seen]
                x = q[lo + i, h].double()
                a = kk @ x * scale
                z = -math.inf if sinks is None else float(sinks[h])
                if not a.numel() and z == -math.inf:
                    continue
                top = max(float(a.max()) if a.numel() else -math.inf, z)
                w = torch.exp(a - top)
                den = w.sum() + math.exp(z - top)
                out[lo + i, h] = (w @ vv) / den if a.numel() else 0.0
                mean[lo + i, h] = (w @ vv.abs()) / den if a.numel() else 0.0
                total_v[lo + i, h] = vv.abs().sum(0) / den if a.numel() else 0.0
                worst[lo + i, h] = float((kk.abs() @ x.abs()).max()) * scale if a.numel() else 0.0
                lse[lo + i, h] = top + torch.log(den)
                count[lo + i, h] = a.numel()
    return {"out": out, "lse": lse, "mean": mean, "worst": worst, "total": total_v, "count": count, "mine": mine}


def bounds(r, dim, cache, out, wide):
    """Bounds of out and lse.

    A score is a sum of `dim` exact products in fp32 (dim + 1 roundings of at most `worst`); q in terms is off by
    2^-22 of its row's largest at most, counted as 2^-21 of `worst` a value of the row.  Scaled, less m, through exp2:
    each of three roundings is at most 2^-23 of the exponent or of the weight; running factors add as many again a
    piece, counted with the sums.  A weight's relative error meets numerator and denominator: twice.  It is rounded to
    the cache's type, u (in terms: 2^-21), and lost below that type's least step, which the sums see as `total`.
    Numerator and denominator are fp32 sums of `count` + 64 terms.  The output rounds once."""
    u = 2.0 ** -21 if wide else EPS[cache] * 1.001
    score = r["worst"] * ((dim + 8) * 2.0 ** -24 + (dim * 2.0 ** -21 if wide else 0.0)) + r["worst"] * 2.0 ** -22 + 2.0 ** -21
    sums = (r["count"] + 64) * 2.0 ** -23
    rel = (u + 2 * score + sums)[..., None]
    tol = r["mean"] * rel + r["total"] * 2.0 ** (-24 if cache is torch.float16 else -125)
    tol = tol + (r["out"].abs() + tol) * EPS[out] * 1.001 + TINY[out]
    return tol, score + sums + 2.0 ** -22 * r["lse"].abs().nan_to_num(0, 0, 0) + 2.0 ** -21


# --- the pool, sequence by sequence -------------------------------------------------

class Pool:
    """What the bookkeeping calls do, said in steps: lists of pages, and the pages' contents as objects."""

    def __init__(self, n_seq, max_pages, n_pages, size):
        self.pages = [[] for _ in range(n_seq)]
        self.lens = [0] * n_seq
        self.max_pages, self.n_pages, self.size = max_pages, n_pages, size
        self.data = list(range(n_pages))

    def refs(self):
        r = [0] * self.n_pages
        for p in self.pages:
            for x in p:
                r[x] += 1
        return r

    def resize(self, wanted):
        size = self.size
        for s, w in enumerate(wanted):
            if 0 <= w < self.lens[s]:
                self.lens[s] = w
                del self.pages[s][-(-w // size):]
        refs = self.refs()
        free = [p for p in range(self.n_pages) if not refs[p]]
        grows = [w > n and -(-w // size) <= self.max_pages for w, n in zip(wanted, self.lens)]
        part = [self.pages[s][-1] if g and self.lens[s] % size else None for s, g in enumerate(grows)]
        at, todo = 0, []
        for s, w in enumerate(wanted):
            if not grows[s]:
                continue
            page, copied = part[s], False
            if page is not None and refs[page] > 1:
                holders = [o for o in range(len(wanted)) if part[o] == page]
                copied = not (len(holders) == refs[page] and holders[0] == s)
            need = -(-w // size) - len(self.pages[s]) + copied
            if at + need <= len(free) or need == 0:
                todo.append((s, w, free[at:at + need], copied))
            at += need
        before = list(self.data)
        for s, w, got, copied in todo:
            if copied:
                self.data[got[0]] = before[self.pages[s][-1]]
                self.pages[s][-1] = got[0]
                got = got[1:]
            self.pages[s] += got
            self.lens[s] = w

    def fork(self, parents):
        pages, lens = [list(p) for p in self.pages], list(self.lens)
        for s, f in enumerate(parents):
            if f == -1:
                self.pages[s], self.lens[s] = [], 0
            elif 0 <= f < len(parents):
                self.pages[s], self.lens[s] = list(pages[f]), lens[f]

    def compact(self):
        refs = self.refs()
        n = sum(r > 0 for r in refs)
        src = [p for p in range(n, self.n_pages) if refs[p]]
        dst = [p for p in range(n) if not refs[p]]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self.data[b] = self.data[a]
        self.pages = [[to.get(x, x) for x in p] for p in self.pages]

    def arrays(self):
        t = torch.full((len(self.pages), self.max_pages), -1, dtype=torch.int32)
        for s, p in enumerate(self.pages):
            t[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
        refs = self.refs()
        used = [0] * ((self.n_pages + 31) // 32)
        for p, r in enumerate(refs):
            used[p // 32] |= (r > 0) << (p % 32)
        used = torch.tensor(used, dtype=torch.int64).to(torch.int32)
        return t, torch.tensor(self.lens, dtype=torch.int32), torch.tensor(refs, dtype=torch.int32), used
