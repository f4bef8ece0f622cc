"""The inputs of kvbound.py in a paged cache on the device, attended by the library and held to their bounds."""
from __future__ import annotations

import kvbound
from kvref import TYPES
from test_gpu_kv import Batch, attend, gen, within

KINDS = [("f16", "f16", "f16"), ("bf16", "bf16", "bf16"), ("f32", "f16", "f32"), ("f32", "bf16", "f32"),
         ("f16", "bf16", "f16"), ("bf16", "f16", "f32"), ("bf16", "bf16", "f32")]


def many_rows(new, group):
    """Whether a call of these new tokens goes to the kernel of many rows."""
    return sum(new) * group > 16 * len(new)


def check(dev, lens, new, heads, kv, dim, kinds, spread, scale=8.0, power=0, smallest=0, causal=True, window=0, parts=1,
          seed=1):
    """`power`: q times 2^power, the scale over it."""
    x, c, y = kinds
    b = Batch(dev, lens, new, kv, dim, c, seed=seed)
    q, keys, values = kvbound.single(gen(seed + dim), lens, b.rows, heads, kv, dim, c, x, spread, scale, smallest)
    q = (q.double() * 2.0 ** power).to(q.dtype)
    scale = scale * 2.0 ** -power
    for s, n in enumerate(lens):
        for j in range(n):
            b.k[1, int(b.tables[s, j // 16]), :, j % 16] = keys[s][j]
            b.v[1, int(b.tables[s, j // 16]), :, j % 16] = values[s][j]
    b.reload()
    out, lse = attend(b, q, y, scale=scale, causal=causal, window=window)
    wide = not (TYPES[x] == TYPES[c] == TYPES[y])
    many = many_rows(new, heads // kv)
    for s, (n, m) in enumerate(zip(lens, new)):
        if not m:
            continue
        rows = slice(b.starts[s], b.starts[s] + m)
        seen = kvbound.seen_of(n, m, causal, window)
        ref, ref_lse = kvbound.exact(q[rows], keys[s], values[s], seen, scale)
        tol = kvbound.bound(ref, values[s], seen, spread, TYPES[c], TYPES[y], wide, many, parts)
        within(out[rows], ref, tol, f"sequence {s} out")
        within(lse[rows], ref_lse, kvbound.bound_lse(ref_lse, seen, spread, TYPES[c], wide, parts), f"sequence {s} lse")
