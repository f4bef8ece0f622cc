"""Timed cases of the operators of a paged cache of keys and values: rotary positions, writing new tokens into the
cache, attention of a chunk of new tokens (one token or a prompt) over it, and the bookkeeping of its pages.

`run` computes a case in its plain form (elementary torch operations in 32 bits, angles in 64, rounded once at the
end) where `own` is false, and through the library's calls where it is true.  `exact` is the operator's definition in
64 bits.

A cache is a pair of tensors (layers, pages, heads, slots, dim).  Position p of sequence s lies in slot p % slots of
page tables[s, p // slots].  Of `lens[s]` positions the last starts[s + 1] - starts[s] are the new tokens', whose rows
of the activations are starts[s] and following.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# --- cases ---------------------------------------------------------------------

def rope(tok, heads, dim, rot, x="bf16", y="bf16", interleaved=False, scaling="none", far=4096, inverse=False, pad=0):
    """Rotary positions of `tok` rows of `heads` heads, the first `rot` of `dim` values of each, or their gradient."""
    return {"op": "rope", "tok": tok, "heads": heads, "dim": dim, "rot": rot, "x": x, "y": y,
            "interleaved": interleaved, "scaling": scaling, "far": far, "inverse": inverse, "pad": pad}


def append(seqs, new, length, q_heads, heads, dim, rot, x="bf16", cache="bf16", page=16, layers=2, interleaved=False,
           ragged=True):
    """New tokens' keys, rotated, and values into the pages, and their queries rotated."""
    return {"op": "append", "seqs": seqs, "new": new, "length": length, "q_heads": q_heads, "heads": heads,
            "dim": dim, "rot": rot, "x": x, "cache": cache, "page": page, "layers": layers,
            "interleaved": interleaved, "ragged": ragged}


def attend(seqs, new, length, q_heads, heads, dim, x="bf16", cache="bf16", y="bf16", page=16, window=0, sinks=False,
           ragged=True, room=1, causal=True):
    """Attention of each sequence's last tokens over its cached positions; tables of `room` times the pages needed."""
    return {"op": "attend", "seqs": seqs, "new": new, "length": length, "q_heads": q_heads, "heads": heads,
            "dim": dim, "x": x, "cache": cache, "y": y, "page": page, "window": window, "sinks": sinks,
            "ragged": ragged, "room": room, "causal": causal}


def beams(prompts, forks, length, heads, dim, cache="bf16", page=16, layers=24):
    """Prompts forked into `forks` sequences each (their last run's let go first), and a place made for one token."""
    return {"op": "beams", "prompts": prompts, "forks": forks, "length": length, "heads": heads, "dim": dim,
            "cache": cache, "page": page, "layers": layers}


def turnover(seqs, length, heads, dim, cache="bf16", page=16, layers=8):
    """Half of the sequences leave, the others move to the lowest pages, new ones come; and so with the other half."""
    return {"op": "turnover", "seqs": seqs, "length": length, "heads": heads, "dim": dim, "cache": cache,
            "page": page, "layers": layers}


def listed():
    return [
        # one decoded token of the 20B-class network, a quarter of each head rotated: launch latency
        {"name": "rope_token", **rope(1, 64, 96, 24, "f32", "f32")},
        # the gradient of a long prompt's rotation, frequencies stretched for a long context
        {"name": "rope_gradient", **rope(8191, 64, 128, 128, "bf16", "bf16", True, "yarn", 1 << 20, True, 64)},
        # one decoded token of the 20B-class network out of its fp32 QKV row
        {"name": "append_token", **append(1, 1, 1000, 64, 64, 96, 24, "f32", "f16", 16, 2, False, False)},
        # a ragged batch of prompts into pages
        {"name": "append_prompt", **append(7, 2048, 4096, 64, 8, 128, 128, "bf16", "bf16", 16, 2)},
        # one decoded token over a short context: launch latency
        {"name": "attend_token", **attend(1, 1, 1500, 64, 8, 64, "bf16", "bf16", "bf16", 16, 0, True, False, 4)},
        # a decoding batch of ragged contexts
        {"name": "attend_batch", **attend(64, 1, 8192, 64, 8, 64, "bf16", "bf16", "bf16", 16, 0, True, True, 2)},
        # one fp32 token of the 20B-class network over a very long context
        {"name": "attend_long", **attend(1, 1, 131009, 64, 64, 96, "f32", "f16", "f32", 32, 0, False, False)},
        # chunks of prompts over what is cached of them, ragged, the 20B-class heads
        {"name": "attend_chunk", **attend(5, 512, 16384, 64, 64, 96, "f16", "f16", "f16", 16)},
        # a prompt with a sliding window, fp32 activations
        {"name": "attend_window", **attend(3, 4096, 4096, 64, 8, 64, "f32", "bf16", "f32", 16, 128, True)},
        # a whole long prompt
        {"name": "attend_prompt", **attend(1, 8192, 8192, 32, 8, 128, "bf16", "bf16", "bf16", 64, 0, False, False)},
        # a step's bookkeeping of beams over shared prompts
        {"name": "pages_beams", **beams(32, 7, 4000, 8, 64)},
        # a batch that changes by half, pages moved together
        {"name": "pages_turnover", **turnover(48, 4000, 8, 64, "bf16", 16, 8)},
    ]


def spread_over(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw_heads(rng):
    dim = rng.choice([32, 64, 64, 96, 128, 128, 128, 160, 192, 224, 256])
    heads = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    group = rng.choice([g for g in (1, 1, 2, 3, 4, 5, 7, 8, 16) if g * heads <= 64])
    return heads * group, heads, dim


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "attend", "beams", "turnover"])
    kinds = ["f32", "f16", "bf16"]
    q_heads, heads, dim = draw_heads(rng)
    page = rng.choice([1, 8, 16, 16, 16, 32, 64, 128])
    cache = rng.choice(["f16", "bf16"])
    if op == "rope":
        x = rng.choice(kinds)
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
        tok = spread_over(rng, 1, min(32768, 8191 * 64 * 128 // (q_heads * dim)))
        return rope(tok, q_heads, dim, rot, x, rng.choice([x, x, "f32"]), rng.random() < 0.5,
                    rng.choice(["none", "linear", "ntk", "yarn"]), spread_over(rng, 16, 1 << 21), rng.random() < 0.4,
                    rng.choice([0, 0, 64, 3]))
    if op == "append":
        seqs = spread_over(rng, 1, 256)
        new = spread_over(rng, 1, max(1, 14336 // seqs))
        length = new + spread_over(rng, 1, 8192)
        while seqs * (length + page) * heads * dim > 1 << 28:
            length = max(new, length // 2)
            seqs = seqs // 2 + 1
        return append(seqs, new, length, q_heads, heads, dim, rng.choice([dim, dim // 2, dim // 4]),
                      rng.choice(kinds), cache, page, 2, rng.random() < 0.3, rng.random() < 0.7)
    if op == "attend":
        seqs = spread_over(rng, 1, 128)
        new = 1 if rng.random() < 0.4 else spread_over(rng, 1, 4096)
        length = new + spread_over(rng, 1, 65536)
        # what the largest listed ones cost
        while seqs * new * length * q_heads * dim > 8192 * 8192 * 32 * 128 // 2 or \
                seqs * length * heads * dim > 64 * 8192 * 8 * 128 or seqs * new * length * q_heads > 1 << 31:
            seqs, new = seqs // 2 + 1 if seqs > 2 else 1, new * 2 // 3 + 1 if new > 1 else 1
            length = max(new, length * 2 // 3)
        x = rng.choice(kinds)
        return attend(seqs, new, length, q_heads, heads, dim, x, cache, rng.choice([x, x, "f32"]), page,
                      rng.choice([0, 0, 0, 128, spread_over(rng, 1, 4096)]), rng.random() < 0.3, rng.random() < 0.7,
                      rng.choice([1, 1, 3]), rng.random() < 0.9)
    length = spread_over(rng, 3, 4000)
    layers = rng.choice([1, 4, 24])
    page = rng.choice([8, 16, 16, 32, 64])
    if op == "beams":
        prompts, forks = spread_over(rng, 1, 32), rng.choice([1, 2, 3, 7])
        while prompts * (length + (forks + 1) * 2 * page) * heads * dim * layers > 32 * 4000 * 8 * 64 * 24 // 2:
            prompts, layers = prompts * 2 // 3 + 1 if prompts > 2 else 1, layers // 2 + 1 if layers > 2 else 1
            length = length * 2 // 3 + 1
            heads = max(1, heads // 2) if prompts == 1 else heads
        return beams(prompts, forks, length, heads, dim, cache, page, layers)
    seqs = spread_over(rng, 2, 200)
    while seqs * (length + page) * heads * dim * layers > 48 * 4000 * 8 * 64 * 8:
        seqs, layers = seqs * 2 // 3 + 1 if seqs > 2 else 2, layers // 2 + 1 if layers > 2 else 1
        length = length * 2 // 3 + 1
        heads = max(1, heads // 2) if seqs == 2 else heads
    return turnover(seqs, length, heads, dim, cache, page, layers)


# --- inputs ----------------------------------------------------------------------

def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def lengths(case):
    """Each sequence's length and new tokens, the case's own: the longest, or up to it with every length as likely; at
    least its new tokens."""
    n, longest = case["seqs"], case["length"]
    r = torch.Generator().manual_seed(n * 1009 + longest)
    if not case["ragged"]:
        return [longest] * n, [case["new"]] * n
    new = torch.randint((case["new"] + 3) // 4, case["new"] + 1, (n,), generator=r)
    lens = torch.maximum(torch.randint(1, longest + 1, (n,), generator=r), new)
    lens[int(torch.randint(0, n, (1,), generator=r))] = longest
    return lens.tolist(), new.tolist()


def paged(g, lens, page, room=1, spare=3):
    """(tables, number of pages): every sequence's pages at places without order, unmapped entries -1."""
    each = torch.tensor([-(-n // page) for n in lens])
    total = int(each.sum())
    order = torch.randperm(total + spare, generator=g, device=DEV).int()
    width = int(each.max()) * room
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    mapped = torch.arange(width)[None] < each[:, None]
    tables[mapped.to(DEV)] = order[:total]
    return tables, total + spare


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def frequencies(case):
    """Radians a position of each pair, and the factor of the rotated values, in 64 bits (on the host)."""
    half, base, factor, trained = case["rot"] // 2, 10000.0, 8.0, 4096.0
    scaling = case.get("scaling", "none")
    if scaling == "ntk" and half > 1:
        base *= factor ** (2 * half / (2 * half - 2.0))
    f = [base ** (-i / half) for i in range(half)]
    if scaling == "linear":
        f = [v / factor for v in f]
    if scaling != "yarn":
        return f, 1.0
    # pairs that turn 32 times and more within the trained length stay, those below one turn are stretched
    fast, slow = (half * math.log(trained / (t * 2 * math.pi)) / math.log(base) for t in (32.0, 1.0))
    fast, slow = max(math.floor(fast), 0), min(math.ceil(slow), 2 * half - 1)
    slow = slow if slow > fast else fast + 0.001
    keep = [1.0 - min(max((i - fast) / (slow - fast), 0.0), 1.0) for i in range(half)]
    return [v / factor * (1 - k) + v * k for v, k in zip(f, keep)], 0.1 * math.log(factor) + 1.0


def cache_of(g, case, pages):
    shape = (case["layers"] if "layers" in case else 1, pages, case["heads"], case["page"], case["dim"])
    return [torch.randn(shape, generator=g, device=DEV, dtype=FLOATS[case["cache"]]) for _ in range(2)]


def batch_of(g, case):
    lens, new = lengths(case)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    tables, pages = paged(g, lens, case["page"], case.get("room", 1))
    return {"lens": ints(lens), "starts": ints(starts), "tables": tables, "pages": pages, "tok": starts[-1],
            "most_new": max(new), "longest": max(lens)}


def pool_of(lens, width, order, page, n_seq):
    """The pages in `order` to the sequences of `lens`, the others empty: tables, lengths, uses of each page, its bits."""
    tables = torch.full((n_seq, width), -1, dtype=torch.int32)
    each = torch.tensor([-(-n // page) for n in lens])
    total = int(each.sum())
    tables[:len(lens)][torch.arange(width)[None] < each[:, None]] = order[:total].int()
    refs = torch.zeros(order.numel(), dtype=torch.int32)
    refs[order[:total]] = 1
    refs = refs.to(DEV)
    return {"tables": tables.to(DEV), "lens": ints(lens + [0] * (n_seq - len(lens))), "refs": refs, "used": bits(refs)}


def prepare(case, seed):
    g = gen(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("rope", "append"):
        f, s["mscale"] = frequencies(case)
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if op == "rope":
        tok, heads, dim, pad = case["tok"], case["heads"], case["dim"], case["pad"]
        s["x"] = torch.randn(tok, heads * dim + pad, generator=g, device=DEV).to(FLOATS[case["x"]])[:, :heads * dim] \
            .unflatten(1, (heads, dim))
        first = torch.randint(0, max(1, case["far"] - tok), (1,), generator=g, device=DEV)
        s["pos"] = (first + torch.arange(tok, device=DEV)).int()
        s["out"] = torch.zeros(tok, heads, dim, dtype=FLOATS[case["y"]], device=DEV)
    elif op == "append":
        s.update(batch_of(g, case))
        q, kv, dim = case["q_heads"], case["heads"], case["dim"]
        qkv = torch.randn(s["tok"], (q + 2 * kv) * dim, generator=g, device=DEV).to(FLOATS[case["x"]])
        s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, dim)) for t in qkv.split([q * dim, kv * dim, kv * dim], 1))
        s["cache"] = cache_of(g, case, s["pages"])
        s["q_out"] = torch.zeros(s["tok"], q, dim, dtype=FLOATS[case["x"]], device=DEV)
    elif op == "attend":
        s.update(batch_of(g, case))
        s["q"] = torch.randn(s["tok"], case["q_heads"], case["dim"], generator=g, device=DEV).mul_(1.5) \
            .to(FLOATS[case["x"]])
        s["cache"] = cache_of(g, case, s["pages"])
        s["sinks"] = torch.randn(case["q_heads"], generator=g, device=DEV) if case["sinks"] else None
        s["out"] = torch.zeros(s["tok"], case["q_heads"], case["dim"], dtype=FLOATS[case["y"]], device=DEV)
        s["lse"] = torch.zeros(s["tok"], case["q_heads"], device=DEV)
        s["keep"] = {}
    else:
        page, r = case["page"], torch.Generator().manual_seed(case["length"])
        longest = case["length"]
        n = case["prompts"] if op == "beams" else case["seqs"]
        # (the lengths are the case's own)
        lens = torch.randint((longest + 1) // 2, longest + 1, (n,), generator=r).tolist()
        width = -(-(longest + 1) // page) + 2
        total = sum(-(-v // page) for v in lens)
        if op == "beams":
            seqs = n * (1 + case["forks"])
            order = torch.randperm(total + 2 * seqs, generator=torch.Generator().manual_seed(seed))
            s.update(pool_of(lens, width, order, page, seqs))
            # the prompts' own lengths again, their forks let go; whose fork each sequence is; one token more
            s["back"] = ints(lens + [0] * (seqs - n))
            parents = torch.arange(seqs) % n
            s["parents"] = parents.int().to(DEV)
            s["grown"] = ints([lens[i] + 1 for i in parents.tolist()])
        else:
            s.update(pool_of(lens, width, torch.arange(total + 5), page, n))
            first = torch.arange(n) < n // 2
            whole = torch.tensor(lens)
            s["leave"] = [torch.where(m, 0, -1).int().to(DEV) for m in (first, ~first)]
            s["come"] = [torch.where(m, whole, -1).int().to(DEV) for m in (first, ~first)]
        s["cache"] = cache_of(g, case, s["refs"].numel())
        s["keep"] = {}
    return s


# --- the plain forms ---------------------------------------------------------------

def turned(x, pos, freqs, interleaved, mscale, inverse=False):
    """The first values of each head of `x` (rows, heads, dim) turned by their row's position, in 32 bits."""
    half = freqs.numel()
    angle = torch.remainder(pos.double()[:, None] * freqs, 2 * math.pi)
    c, s = (torch.cos(angle) * mscale).float()[:, None], (torch.sin(angle) * mscale).float()[:, None]
    s = -s if inverse else s
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def places(s, page):
    """Each row's position, page and slot."""
    row = torch.arange(s["tok"], device=DEV)
    seq = torch.searchsorted(s["starts"].long(), row, right=True) - 1
    end = s["starts"].long()[seq + 1]
    pos = s["lens"].long()[seq] - end + row
    return pos, s["tables"].long()[seq, pos // page], pos % page


def plain_attend(s):
    case = s["case"]
    kv, dim, page = case["heads"], case["dim"], case["page"]
    group, n_seq, new = case["q_heads"] // kv, case["seqs"], s["most_new"]
    wide = -(-s["longest"] // page)
    at = s["tables"].long()[:, :wide].clamp(min=0)
    k, v = (c[0][at].transpose(1, 2).flatten(2, 3).float() for c in s["cache"])  # (seqs, heads, positions, dim)
    count = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(new, device=DEV)
    row = (s["starts"][:-1].long()[:, None] + i).clamp(max=s["tok"] - 1)
    q = s["q"][row].float().view(n_seq, new, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(n_seq, kv, -1, dim)
    scores = torch.matmul(q, k.transpose(-1, -2)).view(n_seq, kv, group, new, -1).mul_(dim ** -0.5)
    j = torch.arange(wide * page, device=DEV)
    lens = s["lens"].long()[:, None]
    pos = (lens - count[:, None] + i)[..., None]
    seen = j < lens[..., None]
    if case["causal"]:
        seen = seen & (j <= pos)
    if case["window"]:
        seen = seen & (j > pos - case["window"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    sink = s["sinks"].view(1, kv, group, 1, 1) if case["sinks"] else None
    top = torch.maximum(top, sink) if case["sinks"] else top
    p = scores.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    total = total + torch.exp(sink - top) if case["sinks"] else total
    o = torch.matmul(p.view(n_seq, kv, -1, wide * page), v).view(n_seq, kv, group, new, dim)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    there = i < count[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(n_seq, new, -1, dim)[there]
    return o.to(FLOATS[case["y"]]), lse.permute(0, 3, 1, 2).reshape(n_seq, new, -1)[there]


def bits(refs):
    """One bit a page in use, 32 to a word."""
    on = torch.nn.functional.pad((refs > 0).long(), (0, -refs.numel() % 32)).view(-1, 32)
    return (on << torch.arange(32, device=refs.device)).sum(1).to(torch.int32)


def counted(s):
    """Uses of each page and its bits, from the tables."""
    live = s["tables"][s["tables"] >= 0].long()
    s["refs"].copy_(torch.bincount(live, minlength=s["refs"].numel()))
    s["used"].copy_(bits(s["refs"]))


def moved(s, src, dst):
    for c in s["cache"]:
        c[:, dst] = c[:, src]


def plain_fork(s):
    tables, lens = s["tables"][s["parents"].long()], s["lens"][s["parents"].long()]
    s["tables"].copy_(tables)
    s["lens"].copy_(lens)
    counted(s)


def plain_resize(s, wanted):
    """Sequences cut or grown to the `wanted` lengths (-1: as it is): pages let go, then lowest free pages taken in the
    sequences' order; a last page that others hold too is copied before it is grown into, but by its first holder
    where all of them grow."""
    page, tables, lens = s["case"]["page"], s["tables"], s["lens"].long()
    wanted = torch.where(wanted < 0, lens, wanted.long())
    n, width = tables.shape
    col = torch.arange(width, device=DEV)
    have = -(-torch.minimum(lens, wanted) // page)
    tables.masked_fill_(col >= have[:, None], -1)
    counted(s)
    refs = s["refs"].long()
    wide = -(-wanted // page) > width
    grows = (wanted > lens) & ~wide
    last = tables.long().gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    partial = grows & (lens % page > 0)
    last = torch.where(partial, last, refs.numel())
    growing = torch.bincount(last, minlength=refs.numel() + 1)
    seq = torch.arange(n, device=DEV)
    first = torch.full_like(growing, n).scatter_reduce_(0, last, seq, "amin")
    uses = torch.nn.functional.pad(refs, (0, 1))
    copies = partial & (uses[last] > 1) & ~((growing[last] == uses[last]) & (first[last] == seq))
    need = torch.where(grows, -(-wanted // page) - have, 0) + copies
    free = (refs == 0).nonzero().flatten()
    before = need.cumsum(0) - need
    fits = ((before + need <= free.numel()) | (need == 0)) & ~wide
    need = torch.where(fits, need, 0)
    owner = torch.repeat_interleave(seq, need)
    rank = torch.arange(owner.numel(), device=DEV) - (need.cumsum(0) - need)[owner]
    got = free[before[owner] + rank]
    src = last[copies & fits]
    tables[owner, (have - copies.long())[owner] + rank] = got.int()
    moved(s, src, got[(rank == 0) & copies[owner]])
    s["lens"].copy_(torch.where(fits, wanted, lens))
    counted(s)


def plain_compact(s):
    used = s["refs"] > 0
    count = used.sum()
    at = torch.arange(used.numel(), device=DEV)
    src, dst = (used & (at >= count)).nonzero().flatten(), (~used & (at < count)).nonzero().flatten()
    moved(s, src, dst)
    to = at.clone()
    to[src] = dst
    s["tables"].copy_(torch.where(s["tables"] >= 0, to[s["tables"].long().clamp(min=0)].int(), -1))
    counted(s)


def pool_out(s):
    return s["tables"], s["lens"], s["refs"], s["used"], s["cache"][0], s["cache"][1]


def plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        return turned(s["x"], s["pos"], s["freqs"], case["interleaved"], s["mscale"], case["inverse"]) \
            .to(s["out"].dtype)
    if op == "append":
        pos, page, slot = places(s, case["page"])
        k, v = s["cache"]
        layer = case["layers"] - 1
        k[layer, page, :, slot] = turned(s["k"], pos, s["freqs"], case["interleaved"], s["mscale"]).to(k.dtype)
        v[layer, page, :, slot] = s["v"].to(v.dtype)
        return k, v, turned(s["q"], pos, s["freqs"], case["interleaved"], s["mscale"]).to(s["q"].dtype)
    if op == "attend":
        return plain_attend(s)
    if op == "beams":
        plain_resize(s, s["back"])
        plain_fork(s)
        plain_resize(s, s["grown"])
    else:
        plain_resize(s, s["leave"][0])
        plain_compact(s)
        plain_resize(s, s["come"][0])
        plain_resize(s, s["leave"][1])
        plain_compact(s)
        plain_resize(s, s["come"][1])
    return pool_out(s)


# --- the library's calls -------------------------------------------------------------

def library(s):
    import quantized_gemv_gguf_amd as q
    case = s["case"]
    op = case["op"]
    if op in ("rope", "append"):
        turn = q.Rope(s["freqs"], interleaved=case["interleaved"], mscale=s["mscale"])
    if op == "rope":
        q.qgemv_rope(s["x"], s["pos"], turn, s["out"], inverse=case["inverse"])
        return s["out"]
    cache = q.KvCache(*s["cache"])
    if op in ("append", "attend"):
        seqs = q.KvSeqs(s["starts"], s["lens"], s["tables"])
    if op == "append":
        q.qgemv_kv_append(s["k"], s["v"], seqs, cache, case["layers"] - 1, rope=turn, q=s["q"], q_out=s["q_out"])
        return (*s["cache"], s["q_out"])
    if op == "attend":
        # the workspace is kept, as a program that decodes keeps it
        if "work" not in s["keep"]:
            n = q.qgemv_kv_attend_bytes(s["q"], seqs, cache)
            s["keep"]["work"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        q.qgemv_kv_attend(s["q"], seqs, cache, 0, s["out"], scale=case["dim"] ** -0.5, causal=case["causal"],
                          window=case["window"], sinks=s["sinks"], lse=s["lse"], work=s["keep"]["work"])
        return s["out"], s["lse"]
    if "work" not in s["keep"]:
        n = q.qgemv_kv_pool_bytes(*s["tables"].shape, s["refs"].numel())
        s["keep"]["work"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    pool = q.KvPool(s["tables"], s["lens"], s["refs"], s["used"], case["page"], s["keep"]["work"])
    if op == "beams":
        q.qgemv_kv_resize(pool, cache, s["back"])
        q.qgemv_kv_fork(pool, s["parents"])
        q.qgemv_kv_resize(pool, cache, s["grown"])
    else:
        for leave, come in zip(s["leave"], s["come"]):
            q.qgemv_kv_resize(pool, cache, leave)
            q.qgemv_kv_compact(pool, cache)
            q.qgemv_kv_resize(pool, cache, come)
    return pool_out(s)


def run(state):
    return library(state) if own else plain(state)


# --- what a pass cannot do without -----------------------------------------------------

def seen_keys(case):
    """(visible pairs of a query and a key, keys read) of the case, all heads of one; expected where it is ragged."""
    n, new, length, window = case["seqs"], case["new"], case["length"], case["window"]
    if case["ragged"]:
        new, length = max(1.0, new * 5 / 8), max(new * 5 / 8, (length + case["new"] / 4) / 2)
    old = length - new
    each = old + (new + 1) / 2 if case["causal"] else length
    keys = length
    if window:
        each = min(each, window)
        keys = min(length, new + window)
    return n * new * each, n * keys


def work(case):
    op = case["op"]
    dim = case["dim"]
    if op == "rope":
        n = case["tok"] * case["heads"] * dim
        return {"bytes": n * (SIZE[case["x"]] + SIZE[case["y"]]),
                "flops": 3.0 * case["tok"] * case["heads"] * case["rot"]}
    if op == "append":
        tok = case["seqs"] * case["new"] * (0.625 if case["ragged"] else 1.0)
        tok = max(tok, case["seqs"])
        x, c = SIZE[case["x"]], SIZE[case["cache"]]
        return {"bytes": tok * dim * (2 * x * case["q_heads"] + 2 * (x + c) * case["heads"]),
                "flops": 3.0 * tok * case["rot"] * (case["q_heads"] + case["heads"])}
    if op == "attend":
        pairs, keys = seen_keys(case)
        tok = max(case["seqs"], case["seqs"] * case["new"] * (0.625 if case["ragged"] else 1.0))
        return {"bytes": keys * case["heads"] * dim * 2 * SIZE[case["cache"]] +
                tok * case["q_heads"] * dim * (SIZE[case["x"]] + SIZE[case["y"]]),
                "flops": 4.0 * pairs * case["q_heads"] * dim}
    page_bytes = 2 * case["layers"] * case["heads"] * case["page"] * dim * SIZE[case["cache"]]
    mean = 0.75 * case["length"] / case["page"] + 1
    if op == "beams":
        # the tables' rows read and written, the uses; each fork's last page read and written
        seqs = case["prompts"] * case["forks"]
        return {"bytes": seqs * (4 * 4 * mean + 2 * page_bytes * (1 - 1 / case["page"])), "flops": seqs * mean}
    # each half's pages read and written once; tables and uses of all pages
    return {"bytes": case["seqs"] * mean * (2 * page_bytes + 32), "flops": case["seqs"] * mean}


# --- the definition in 64 bits ---------------------------------------------------------

def exact_turn(x, pos, freqs, interleaved, mscale, inverse):
    """Pairs as complex numbers, times mscale e^(i angle)."""
    half = freqs.numel()
    x = x.double()
    at = torch.arange(half, device=DEV)
    re, im = (2 * at, 2 * at + 1) if interleaved else (at, at + half)
    angle = pos.double()[:, None, None] * freqs
    z = torch.complex(x[..., re], x[..., im]) * torch.polar(torch.full_like(angle, mscale), -angle if inverse else angle)
    y = x.clone()
    y[..., re], y[..., im] = z.real, z.imag
    return y


def exact_attend(s):
    """One sequence and head of the cache at a time."""
    case = s["case"]
    kv, dim = case["heads"], case["dim"]
    group = case["q_heads"] // kv
    out = torch.zeros(s["tok"], case["q_heads"], dim, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["tok"], case["q_heads"], dtype=torch.float64, device=DEV)
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for i, n in enumerate(lens):
        lo, hi = starts[i], starts[i + 1]
        at = s["tables"][i, :-(-n // case["page"])].long()
        j, p = torch.arange(n, device=DEV), torch.arange(n - (hi - lo), n, device=DEV)[:, None]
        hidden = torch.zeros(hi - lo, n, dtype=torch.bool, device=DEV)
        if case["causal"]:
            hidden |= j > p
        if case["window"]:
            hidden |= j <= p - case["window"]
        for h in range(kv):
            k, v = (c[0, at, h].flatten(0, 1)[:n].double() for c in s["cache"])
            for m in range(h * group, (h + 1) * group):
                a = (s["q"][lo:hi, m].double() @ k.T / math.sqrt(dim)).masked_fill_(hidden, -math.inf)
                if case["sinks"]:
                    a = torch.cat([a, s["sinks"][m].double().expand(hi - lo, 1)], 1)
                lse[lo:hi, m] = torch.logsumexp(a, 1)
                out[lo:hi, m] = torch.exp(a - lse[lo:hi, m, None])[:, :n] @ v
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return exact_turn(s["x"], s["pos"], s["freqs"], case["interleaved"], s["mscale"], case["inverse"])
    if op == "append":
        k, v = (c.double() for c in s["cache"])
        turn = [exact_turn(t, places(s, 1 << 30)[0], s["freqs"], case["interleaved"], s["mscale"], False)
                for t in (s["k"], s["q"])]
        starts, lens, size = s["starts"].tolist(), s["lens"].tolist(), case["page"]
        layer = case["layers"] - 1
        for i, n in enumerate(lens):
            p = torch.arange(n - (starts[i + 1] - starts[i]), n, device=DEV)
            at = s["tables"][i].long()[p // size]
            k[layer, at, :, p % size] = turn[0][starts[i]:starts[i + 1]]
            v[layer, at, :, p % size] = s["v"][starts[i]:starts[i + 1]].double()
        return k, v, turn[1]
    if op == "attend":
        return exact_attend(s)
    return None
