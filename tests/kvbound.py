"""Inputs for the paged cache's attention that show every weight by itself, their 64-bit results, and relative bounds.

Key j has one value that is not 0, and so has value j: a score is scale * q[a(j)] * k_j, one product, and an output is
the weights of the keys whose value lies there, over their sum.  Everything that is summed is positive, so errors are
relative to each output: a weight far below the row's largest has to be as exact as its share of the bound says, and
rounding in the products of the matrix instructions hides nothing.  The q values of a row lie up to 2^15 apart."""
from __future__ import annotations

import math

import torch

from kvref import EPS, TINY, TYPES

WIDE = {torch.float16: 2, torch.bfloat16: 3}       # terms where the call's types differ
SMALLEST_Q = 15                                    # a row's q values: 2^-15 to 1 of the largest


def single(g, lens, rows, heads, kv, dim, kind, x, spread, scale, smallest=SMALLEST_Q):
    """(q (rows, heads, dim) of type x, k and v of each sequence (n, kv, dim) of `kind`): q values from 2^-smallest to 1
    of the row's largest, scores in [-spread, 0], the first two keys' 0, values in [2048, 4096)."""
    low = torch.randint(0, smallest + 1, (dim,), generator=g)
    low[0] = 0
    q = (1 + torch.rand(rows, heads, dim, generator=g)) * 2.0 ** -low.float()
    q = q.to(TYPES[x])
    keys, values = [], []
    for n in lens:
        at = torch.cat([torch.randperm(dim, generator=g) for _ in range(n // dim + 1)])[:n]
        to = torch.cat([torch.randperm(dim, generator=g) for _ in range(n // dim + 1)])[:n]
        k, v = (torch.zeros(n, kv, dim, dtype=TYPES[kind]) for _ in range(2))
        c = torch.rand(n, kv, generator=g) * (spread / scale / 2)
        c[:2] = 0.0
        j = torch.arange(n)[:, None]
        h = torch.arange(kv)[None]
        k[j, h, at[:, None]] = (-c * 2.0 ** low[at][:, None].float()).to(TYPES[kind])
        v[j, h, to[:, None]] = ((1 + torch.rand(n, kv, generator=g)) * 2048).to(TYPES[kind])
        keys.append(k)
        values.append(v)
    return q, keys, values


def seen_of(n, new, causal=True, window=0):
    """(new, n) truth values: what each of a sequence's last rows sees."""
    j, p = torch.arange(n)[None], torch.arange(n - new, n)[:, None]
    seen = torch.ones(new, n, dtype=torch.bool)
    if causal:
        seen &= j <= p
    if window:
        seen &= j > p - window
    return seen


def exact(q, k, v, seen, scale):
    """One sequence: (out, lse) in 64 bits, q (new, heads, dim)."""
    group = q.shape[1] // k.shape[1]
    kk, vv = (t.double().repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))  # (heads, n, dim)
    s = torch.matmul(q.double().transpose(0, 1), kk.transpose(1, 2)) * scale            # (heads, new, n)
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - top)
    total = w.sum(-1, keepdim=True)
    return (torch.matmul(w, vv) / total).transpose(0, 1), (top + total.log())[..., 0].T


def bound(out, v, seen, spread, kind, y, wide, many, parts=1):
    """Bound of one sequence's outputs.

    A score's errors, relative to it: its q value in NT terms (2^-22 and, of the row's largest, 2^-39 in fp16, whose
    least step is 2^-24 where the row's largest is 2^14 and more, so up to 2^-24 of a value 2^-15 as large; 2^-24 in
    bf16), the sum of NT products and the scale (2^-23 for each sum and the scale).  It is at most `spread`, and the
    distance from the largest rounds once more, 2^-24 of at most 1.5 `spread`; exp2 is off by 2^-23.  The weight is taken
    in terms (2^-22, 2^-24) or rounded once, and lost below half the least step of its type: with fp16's largest weight
    of a row at 2^15 (few rows) or at least 2^7 (many) that is 2^-40 and 2^-32 of the largest.  Each of these meets the
    sum of the weights too.  Sums of positive values round by 2^-24 for each addition on the longest way: of the
    weights, half the keys in a lane; of the products, the terms of the keys whose value lies there; then waves, parts
    and the factors as the maximum grows, 8 and the parts for each.  (Adding zeros is exact.)"""
    terms = WIDE[kind] if wide else 1
    half_step = {(torch.float16, True): 2.0 ** -22, (torch.bfloat16, True): 2.0 ** -24}.get((kind, wide), EPS[kind])
    q_term = (2.0 ** -22 + 2.0 ** -23 if kind is torch.float16 else 2.0 ** -24) if wide else 0.0
    score = spread * (q_term + terms * 2.0 ** -23 + 1.5 * 2.0 ** -24) + 2.0 ** -23
    n, dim = seen.shape[1], out.shape[2]
    rel = half_step + 2 * score + (n / 2 + terms * -(-n // dim) + 2 * (8 + parts)) * 2.0 ** -24
    # (what is lost of each weight, over the sum of the weights: at least 1)
    lost = (2.0 ** -32 if many else 2.0 ** -40) if kind is torch.float16 else 2.0 ** -120
    group = out.shape[1] // v.shape[1]
    vv = v.double().repeat_interleave(group, 1).transpose(0, 1)
    gone = torch.matmul(seen.double()[None].expand(vv.shape[0], -1, -1), vv).transpose(0, 1) * lost * 1.01
    tol = out * rel * 1.01 + gone
    return tol + (out + tol) * EPS[y] * 1.001 + TINY[y]


def bound_lse(lse, seen, spread, kind, wide, parts=1):
    """Bound of the log of the sum of the weights: the scores', the sum's, and its own rounding beside a running maximum
    that may be 16 from the largest (in powers of 2)."""
    terms = WIDE[kind] if wide else 1
    q_term = (2.0 ** -22 + 2.0 ** -23 if kind is torch.float16 else 2.0 ** -24) if wide else 0.0
    score = spread * (q_term + terms * 2.0 ** -23 + 1.5 * 2.0 ** -24) + 2.0 ** -23
    return score + (seen.shape[1] / 2 + 16 + 2 * parts) * 2.0 ** -24 + (lse.abs() + spread + 32) * 2.0 ** -22


def terms_of(x, kind, n):
    left, out = x.float(), []
    for _ in range(n):
        t = left.to(kind)
        out.append(t.float())
        left = left - out[-1]
    return out


def emulated(q, k, v, seen, scale, kind, q_terms, w_terms, top_weight=0, q_top=0):
    """The kernels' arithmetic on the CPU: q in `q_terms` terms, its row's largest value at 2^q_top where its type is
    fp16, weights in `w_terms` terms with the row's largest at 2^top_weight, sums in 32 bits."""
    group = q.shape[1] // k.shape[1]
    kk, vv = (t.float().repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))
    x = q.float().transpose(0, 1)
    e = torch.zeros(x.shape[:2] + (1,))
    if kind is torch.float16 and q_terms + w_terms > 2:
        e = torch.floor(torch.log2(x.abs().amax(-1, keepdim=True))) - q_top
    s = sum(torch.matmul(t, kk.transpose(1, 2)) for t in terms_of(x * 2.0 ** -e, kind, q_terms))
    s = (s * (torch.tensor(scale * 1.4426950408889634).float() * 2.0 ** e)).masked_fill(~seen, -math.inf)
    p = torch.exp2(s - (s.amax(-1, keepdim=True) - top_weight))
    o = sum(torch.matmul(t, vv) for t in terms_of(p, kind, w_terms))
    return (o / p.sum(-1, keepdim=True)).transpose(0, 1)
