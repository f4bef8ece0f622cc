"""Plain 64-bit forms of the MXFP4 prompt operators, for the tests: numpy, from
the formulas, sharing nothing with the library or the oracle.

Bounds.  A product's terms are exact (an E2M1 weight times a power of two, an
activation as an exact sum of bf16 terms, or another such weight).  One matrix
instruction adds 32 of them (128 for 4-bit activations) to the running fp32 sum;
counting four roundings of at most a whole fp32 step (2^-23) of the running
sum's bound S = sum |x w| per instruction gives

    |y - ref| <= 4 * steps * 2^-23 * S,   steps = terms * k / 32  (k / 128)

and storing y adds half a step of its type.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# values below this are subnormal in the type: half a step is absolute there
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
STEPS = {"f32": 3 / 32, "f16": 2 / 32, "bf16": 1 / 32, "mxfp4": 1 / 128}


def quantize(x):
    """MXFP4 blocks (rows, k / 32 * 17) of float64 rows, by search over the grid."""
    n, k = x.shape
    b = np.asarray(x, np.float64).reshape(n, k // 32, 32)
    a = np.abs(b).max(-1)
    with np.errstate(all="ignore"):
        e = np.where(a > 0, np.frexp(a)[1] - 1 - 2 + 127, 0)
    e = np.clip(e, 0, 254).astype(np.int64)
    fine = np.isfinite(a)
    with np.errstate(all="ignore"):
        m = np.abs(b) * np.ldexp(1.0, 127 - e)[..., None]
    # of the grid's values the nearest, of two equally near the even code
    d = np.abs(np.where(np.isfinite(m), m, 0.0)[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    near = d == best
    code = np.where(near[..., ::2].any(-1), near[..., ::2].argmax(-1) * 2, near.argmax(-1))
    code = code | (np.signbit(b).astype(np.int64) << 3)
    code = np.where(fine[..., None], code, 0)
    e = np.where(fine, e, 255)
    out = np.empty((n, k // 32, 17), np.uint8)
    out[..., 0] = e
    out[..., 1:] = code[..., :16] | (code[..., 16:] << 4)
    return out.reshape(n, -1)


def values(blocks, k):
    """float64 values of rows of blocks."""
    b = np.asarray(blocks).reshape(-1, k // 32, 17)
    q = b[..., 1:].astype(np.int64)
    code = np.concatenate([q & 15, q >> 4], -1)
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    e = b[..., :1].astype(np.int64)
    v = v * np.where(e == 255, np.nan, np.ldexp(1.0, np.minimum(e, 254) - 127))
    return v.reshape(-1, k)


def random_blocks(rng, rows, k, lo=117, hi=124):
    b = rng.integers(0, 256, (rows, k // 32, 17), dtype=np.uint8)
    b[..., 0] = rng.integers(lo, hi, (rows, k // 32))
    return b.reshape(rows, -1)


def product(x, w, kind):
    """(x W^T, the bound on the library's fp32 sums)."""
    ref = x @ w.T
    s = np.abs(x) @ np.abs(w).T
    return ref, 4 * np.ceil(STEPS[kind] * x.shape[1]) * 2.0 ** -23 * s


def swiglu(g, dg, u, du):
    """silu(g) u and its bound from those of g and u: |silu'| < 1.1, and the hardware exp2 and reciprocal
    cost (|g| + 8) 2^-24 of the value."""
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    h = s * u
    return h, 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + (np.abs(g) + 8) * 2.0 ** -24 * np.abs(h)


def sort(ids, n_expert):
    """(offsets, slots, pos) of the stable sort of the slots by expert."""
    flat = [int(i) for i in np.asarray(ids).ravel()]
    order = sorted((i for i in range(len(flat)) if 0 <= flat[i] < n_expert), key=lambda i: flat[i])
    offsets = [sum(0 <= f < e for f in flat) for e in range(n_expert)] + [len(order)]
    pos = np.full(len(flat), -1)
    pos[order] = np.arange(len(order))
    return np.array(offsets), np.array(order + [-1] * (len(flat) - len(order)), np.int64), pos.reshape(np.shape(ids))


def near(got, ref, bound, kind, what=""):
    """Every output within the bound plus half a step of its type; NaN and infinities in the same places."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{what}: infinities"
    b = np.broadcast_to(bound, ref.shape)[fine]
    allowed = b + HALF[kind] * (np.abs(ref[fine]) + b) + TINY[kind]
    err = np.abs(got[fine] - ref[fine])
    assert np.all(err <= allowed), (f"{what}: {np.sum(err > allowed)} of {err.size} beyond the bound, worst "
                                    f"{np.max(err / allowed):.3g} times it")
