"""Timed cases of the MXFP4 prompt operators: quantisation, products over any
number of tokens, products of tokens sorted by expert, and the sort itself with
the way back and its gradient.

`run` computes a case in its plain form (elementary torch operations in 32 bits,
rounded once at the end) where `own` is false, and through the library's calls
where it is true.  `exact` is the operator's definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "mxfp4": 17 / 32}


# --- cases ---------------------------------------------------------------------

def quant(n, k, x="bf16", out="bf16", pad=0, spread=1.0):
    """Rows quantised to MXFP4 blocks, and the values the blocks stand for."""
    return {"op": "quant", "n": n, "k": k, "x": x, "out": out, "pad": pad, "spread": spread}


def rows(tok, n, k, x="bf16", y="bf16", pair=False, pad=0, skip=0):
    """y = x W^T (or the SwiGLU pair of two W) for `tok` tokens; rows [skip, skip + n) of W."""
    return {"op": "rows", "tok": tok, "n": n, "k": k, "x": x, "y": y, "pair": pair, "pad": pad, "skip": skip}


def experts(tok, sel, experts, n, k, x="bf16", y="bf16", pair=False, gathered=True, dropped=0.0):
    """The experts' products of tokens sorted by expert."""
    return {"op": "experts", "tok": tok, "sel": sel, "experts": experts, "n": n, "k": k, "x": x, "y": y,
            "pair": pair, "gathered": gathered, "dropped": dropped}


def route(tok, sel, experts, k, x="bf16", y="f32", dropped=0.0, grad=False):
    """Tokens sorted by expert and back with weights applied, or the gradient of that."""
    return {"op": "route", "tok": tok, "sel": sel, "experts": experts, "k": k, "x": x, "y": y,
            "dropped": dropped, "grad": grad}


def listed():
    return [
        # one decoded token's activations before a 4-bit product: launch latency
        {"name": "quant_token", **quant(1, 2880, "f32", "f32")},
        # a prompt's activations, the 20B-class hidden width, with a few loud channels' spread
        {"name": "quant_prompt", **quant(8192, 6144, "bf16", "bf16", 0, 4.0)},
        # an odd number of rows in a padded buffer
        {"name": "quant_strided", **quant(1021, 2880, "f16", "f16", 40)},
        # a prompt through the 20B-class up projection, activations in 4 bits
        {"name": "rows_prompt_mxfp4", **rows(4096, 24576, 6144, "mxfp4", "bf16")},
        # a ragged prompt through a gate/up pair of the 11008/4096 network
        {"name": "rows_pair_bf16", **rows(333, 11008, 4096, "bf16", "bf16", True)},
        # a few fp32 tokens of a decoding batch, the down projection's long k
        {"name": "rows_few_f32", **rows(23, 4096, 11008, "f32", "f32", False, 8, 0)},
        # one decoded token: 4 of 128 experts, gate/up pair, ids on the device
        {"name": "experts_token", **experts(1, 4, 128, 2880, 2880, "f32", "f32", True)},
        # a prompt through gate/up of 4 of 128 experts, activations in 4 bits
        {"name": "experts_prompt_mxfp4", **experts(4096, 4, 128, 2880, 2880, "mxfp4", "bf16", True)},
        # the way down of a shorter ragged prompt, rows already in the experts' order, some dropped
        {"name": "experts_down_bf16", **experts(1000, 4, 128, 2880, 2880, "bf16", "bf16", False, False, 0.03)},
        # the routing of one decoded token
        {"name": "route_token", **route(1, 4, 128, 2880, "f32", "f32")},
        # the routing of a long prompt
        {"name": "route_prompt", **route(8192, 4, 128, 2880, "bf16", "bf16")},
        # the gradient of a training step's routing, some slots dropped
        {"name": "route_gradient", **route(4097, 4, 128, 2880, "bf16", "f32", 0.02, True)},
    ]


def spread_over(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def width(rng, lo=64, hi=8192):
    """A number of inputs: whole blocks of 32."""
    return 32 * spread_over(rng, lo // 32, hi // 32)


def draw(rng):
    op = rng.choice(["quant", "rows", "rows", "experts", "experts", "route"])
    x = rng.choice(["f32", "f16", "bf16"])
    y = rng.choice(["f32", "f16", "bf16"])
    if op == "quant":
        k = width(rng)
        return quant(spread_over(rng, 1, (1 << 25) // k), k, x, rng.choice(["f32", "bf16", x]),
                     rng.choice([0, 0, 3, 32]), rng.choice([1.0, 4.0]))
    if op == "rows":
        tok, k, n = spread_over(rng, 1, 4096), width(rng, 64, 16384), spread_over(rng, 16, 16384)
        # a plain product of the largest listed size is what a draw may cost
        while tok * k * n > 4096 * 6144 * 8192:
            tok = tok // 2 + 1
        return rows(tok, n, k, rng.choice([x, "mxfp4"]), y, rng.random() < 0.4, rng.choice([0, 0, 8, 5]),
                    rng.choice([0, 0, 7]))
    sel = rng.choice([1, 2, 4, 4, 6, 8])
    e = spread_over(rng, sel, 160)
    dropped = rng.choice([0.0, 0.0, 0.1])
    if op == "experts":
        k, n = width(rng, 64, 4096), spread_over(rng, 16, 4096)
        tok = spread_over(rng, 1, 4096)
        while tok * sel * k * n > 4096 * 4 * 2880 * 2880 or e * k * n > 128 * 2880 * 2880:
            tok, n, k = tok * 3 // 4 + 1, n * 3 // 4 + 1, max(64, k * 3 // 4 // 32 * 32)
        return experts(tok, sel, e, n, k, rng.choice([x, "mxfp4"]), y, rng.random() < 0.5, rng.random() < 0.5,
                       dropped)
    k = rng.choice([width(rng), spread_over(rng, 3, 8192)])
    return route(spread_over(rng, 1, min(32768, (1 << 26) // (k * sel))), sel, e, k, x, y, dropped, rng.random() < 0.5)


# --- the blocks, for the inputs and the plain forms ------------------------------

# values of the codes 0..15 (sign, two exponent bits, one mantissa bit)
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def pow2(e, dtype=torch.float64):
    """2^e for whole e, exactly (in 64 bits: the reciprocal of a scale passes fp32's normal range)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64).to(dtype)


def quantised(x):
    """(scale bytes, codes' magnitudes and signs as values) of the blocks of 32 along the last axis of `x`."""
    v = x.float().unflatten(-1, (-1, 32))
    a = v.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, (torch.frexp(a)[1] + 124).clamp(0, 254), 0)
    s = v.double() * pow2(127 - e)
    m = s.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=6.0)
    e = torch.where(torch.isfinite(a), e, 255)
    return e, torch.copysign(m, s)


def packed(x):
    """The rows of `x` as MXFP4 blocks: (rows, k / 32 * 17) bytes."""
    e, v = quantised(x)
    m = v.abs()
    code = (m * 2).clamp(max=4) + (m > 2) + (m > 3) + (m > 4)
    code = code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    b = torch.cat([e.to(torch.uint8), code[..., :16] | (code[..., 16:] << 4)], -1)
    return b.flatten(-2).contiguous()


def values(blocks, k, dtype=torch.float32):
    """The values of rows of MXFP4 blocks: a table of the codes, times the scale."""
    b = blocks.view(*blocks.shape[:-1], k // 32, 17)
    q = b[..., 1:]
    code = torch.cat([q & 15, q >> 4], -1)
    table = torch.tensor(E2M1, dtype=dtype, device=b.device)
    v = table.index_select(0, code.flatten().int()).view(code.shape)
    e = b[..., :1].int()
    s = torch.where(e < 255, pow2(e - 127, dtype), math.nan)
    return v.mul_(s).flatten(-2)


# --- inputs ----------------------------------------------------------------------

def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def activations(g, n, k, dtype, spread=1.0, pad=0):
    """Rows about 1, with per-channel loudness of `spread` (a view of a wider buffer if `pad`)."""
    x = torch.randn(n, k + pad, generator=g, device=DEV)
    if spread != 1.0:
        loud = torch.rand(k + pad, generator=g, device=DEV) * 2 - 1
        x.mul_(spread ** loud)
    return x.to(FLOATS[dtype])[:, :k]


def weights(g, n, k):
    """n rows of k MXFP4 weights of deviation 1 / sqrt(k), in pieces that bound the temporaries."""
    out = torch.empty(n, k // 32 * 17, dtype=torch.uint8, device=DEV)
    piece = max(1, (1 << 25) // k)
    for i in range(0, n, piece):
        m = min(piece, n - i)
        out[i:i + m] = packed(torch.randn(m, k, generator=g, device=DEV).mul_(k ** -0.5))
    return out


def choices(g, case):
    """Each token's experts, distinct, some experts more popular than others; -1 where a slot is dropped."""
    tok, sel, e = case["tok"], case["sel"], case["experts"]
    liking = torch.randn(tok, e, generator=g, device=DEV) + 0.5 * torch.randn(e, generator=g, device=DEV)
    ids = liking.topk(sel, 1)[1].int()
    if case["dropped"]:
        ids[torch.rand(tok, sel, generator=g, device=DEV) < case["dropped"]] = -1
    return ids.contiguous()


def sorted_slots(ids, n_expert):
    """(offsets, slots, pos) of the stable sort of the slots by expert, dropped ones behind the last."""
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < n_expert), flat, n_expert)
    order = torch.argsort(key, stable=True)
    count = (key[:, None] == torch.arange(n_expert, device=ids.device)).sum(0) if flat.numel() * n_expert < 1 << 28 \
        else torch.bincount(key, minlength=n_expert + 1)[:n_expert]
    offsets = torch.zeros(n_expert + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = count.cumsum(0)
    there = key[order] < n_expert
    slots = torch.where(there, order, -1)
    pos = torch.empty_like(order)
    pos[order] = torch.where(there, torch.arange(order.numel(), device=ids.device), -1)
    return offsets.int(), slots.int(), pos.int().view(ids.shape)


def blocks_or_floats(x, kind):
    return packed(x) if kind == "mxfp4" else x


def prepare(case, seed):
    g = gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "quant":
        n, k = case["n"], case["k"]
        s["x"] = activations(g, n, k, case["x"], case["spread"], case["pad"])
        s["blocks"] = torch.zeros(n, k // 32 * 17, dtype=torch.uint8, device=DEV)
        s["out"] = torch.zeros(n, k, dtype=FLOATS[case["out"]], device=DEV)
    elif op == "rows":
        tok, n, k = case["tok"], case["n"], case["k"]
        kind = "f32" if case["x"] == "mxfp4" else case["x"]
        s["x"] = blocks_or_floats(activations(g, tok, k, kind, 2.0, 0 if case["x"] == "mxfp4" else case["pad"]),
                                  case["x"])
        s["w"] = [weights(g, n + case["skip"], k) for _ in range(2 if case["pair"] else 1)]
        s["y"] = torch.zeros(tok, n + case["pad"], dtype=FLOATS[case["y"]], device=DEV)[:, :n]
    elif op == "experts":
        tok, sel, e, n, k = case["tok"], case["sel"], case["experts"], case["n"], case["k"]
        ids = choices(g, case)
        s["offsets"], s["slots"], _ = sorted_slots(ids, e)
        # what the plain form needs of the sort: the experts that some token chose, each sorted row's expert
        # among them and its place in it, the fullest expert
        counts = s["offsets"][1:] - s["offsets"][:-1]
        s["chosen"] = counts.nonzero().flatten()
        s["rows"], s["most"] = int(s["offsets"][-1]), int(counts.max())
        expert = ids.flatten()[s["slots"][:s["rows"]].long()].long()
        s["place"] = torch.arange(s["rows"], device=DEV) - s["offsets"].long()[expert]
        s["expert"] = torch.searchsorted(s["chosen"], expert)
        kind = "f32" if case["x"] == "mxfp4" else case["x"]
        s["x"] = blocks_or_floats(activations(g, tok if case["gathered"] else tok * sel, k, kind, 2.0), case["x"])
        s["w"] = [weights(g, e * n, k) for _ in range(2 if case["pair"] else 1)]
        s["y"] = torch.zeros(tok * sel, n, dtype=FLOATS[case["y"]], device=DEV)
    else:
        tok, sel, e, k = case["tok"], case["sel"], case["experts"], case["k"]
        s["ids"] = choices(g, case)
        w = torch.rand(tok, sel, generator=g, device=DEV) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        x, y = FLOATS[case["x"]], FLOATS[case["y"]]
        whole = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=DEV)  # noqa: E731
        if case["grad"]:
            _, _, s["pos"] = sorted_slots(s["ids"], e)
            s["dout"] = torch.randn(tok, k, generator=g, device=DEV).to(y)
            s["y"] = torch.randn(tok * sel, k, generator=g, device=DEV).to(x)
            s["dy"] = torch.zeros(tok * sel, k, dtype=x, device=DEV)
            s["dw"] = torch.zeros(tok, sel, device=DEV)
            s["dx"] = torch.zeros(tok, k, dtype=y, device=DEV)
        else:
            s["x"] = torch.randn(tok, k, generator=g, device=DEV).to(x)
            s["y"] = torch.randn(tok * sel, k, generator=g, device=DEV).to(x)
            s["offsets"], s["slots"], s["pos"] = whole(e + 1), whole(tok * sel), whole(tok, sel)
            s["xs"] = torch.zeros(tok * sel, k, dtype=x, device=DEV)
            s["out"] = torch.zeros(tok, k, dtype=y, device=DEV)
    return s


# --- the plain forms ---------------------------------------------------------------

def silu_times(g, u):
    return g / (1 + torch.exp(-g)) * u


def product(x, ws, k, pair):
    """x W^T, or silu(x G^T) * (x U^T), along the last two axes, in 32 bits."""
    out = [torch.matmul(x, values(w, k).transpose(-1, -2)) for w in ws]
    return silu_times(*out) if pair else out[0]


def plain(s):
    case = s["case"]
    op, k = case["op"], case["k"]
    if op == "quant":
        e, v = quantised(s["x"])
        scale = torch.where(e < 255, pow2(e - 127), math.nan)
        return (v * scale).flatten(-2).to(FLOATS[case["out"]])
    if op == "rows":
        x = values(s["x"], k) if case["x"] == "mxfp4" else s["x"].float()
        return product(x, [w[case["skip"]:] for w in s["w"]], k, case["pair"]).to(s["y"].dtype)
    if op == "experts":
        tok, sel, e, n = case["tok"], case["sel"], case["experts"], case["n"]
        x = values(s["x"], k) if case["x"] == "mxfp4" else s["x"].float()
        at = s["slots"][:s["rows"]].long() // sel if case["gathered"] else torch.arange(s["rows"], device=DEV)
        xs = torch.zeros(s["chosen"].numel(), s["most"], k, device=DEV)
        xs[s["expert"], s["place"]] = x[at]
        h = product(xs, [w.view(e, n, -1)[s["chosen"]] for w in s["w"]], k, case["pair"])
        y = torch.zeros_like(s["y"])
        y[:s["rows"]] = h[s["expert"], s["place"]].to(y.dtype)
        return y
    there = (s["pos"] if case["grad"] else s["ids"]) >= 0
    if case["grad"]:
        pos = s["pos"].long().clamp(min=0)
        dout, yr = s["dout"].float()[:, None], s["y"].float()[pos]
        dw = torch.where(there, (dout * yr).sum(-1), 0.0)
        dys = (s["w"][..., None] * dout).to(s["y"].dtype)
        dy = torch.zeros_like(s["y"])
        dy[s["pos"][there].long()] = dys[there]
        dx = (torch.where(there[..., None], dy[pos].float(), 0.0)).sum(1).to(s["dout"].dtype)
        return dy, dw, dx
    offsets, slots, pos = sorted_slots(s["ids"], case["experts"])
    xs = torch.where(slots[:, None] >= 0, s["x"][slots.long().clamp(min=0) // case["sel"]], 0)
    out = torch.where(there[..., None], s["w"][..., None] * s["y"][pos.long().clamp(min=0)].float(), 0.0).sum(1)
    return offsets, slots, pos, xs, out.to(s["out"].dtype)


# --- the library's calls -------------------------------------------------------------

def library(s):
    import quantized_gemv_gguf_amd as q
    case = s["case"]
    op, k = case["op"], case["k"]

    def matrix(blocks):
        return q.Matrix(blocks, q.MXFP4, blocks.shape[0], k)

    if op == "quant":
        m = matrix(s["blocks"])
        q.qgemv_mx_quantize(s["x"], m)
        q.qgemv_mx_dequantize(m, 0, case["n"], s["out"])
        return s["out"]
    if op in ("rows", "experts"):
        x = matrix(s["x"]) if case["x"] == "mxfp4" else s["x"]
        ws = [matrix(w) for w in s["w"]]
    if op == "rows":
        window = (case["skip"], case["skip"] + case["n"])
        call = q.qgemv_rows_mx_swiglu if case["pair"] else q.qgemv_rows_mx
        call(*ws, *window, x, s["y"])
        return s["y"]
    if op == "experts":
        call = q.qgemv_expert_mx_swiglu if case["pair"] else q.qgemv_expert_mx
        if case["gathered"]:
            call(*ws, case["experts"], x, s["offsets"], s["y"], slots=s["slots"], n_sel=case["sel"])
        else:
            call(*ws, case["experts"], x, s["offsets"], s["y"])
        return s["y"]
    if case["grad"]:
        q.qgemv_expert_combine_grad(s["dout"], s["y"], s["pos"], s["w"], s["dy"], s["dw"])
        q.qgemv_expert_combine(s["dy"], s["pos"], s["dx"])  # the gather's gradient
        return s["dy"], s["dw"], s["dx"]
    q.qgemv_expert_sort(s["ids"], case["experts"], s["offsets"], s["slots"], s["pos"])
    q.qgemv_expert_gather(s["x"], s["slots"], case["sel"], s["xs"])
    q.qgemv_expert_combine(s["y"], s["pos"], s["out"], w=s["w"])
    return s["offsets"], s["slots"], s["pos"], s["xs"], s["out"]


def run(state):
    return library(state) if own else plain(state)


# --- what a pass cannot do without -----------------------------------------------------

def touched(case):
    """Experts that some token chose, expected over uniform choices."""
    e = case["experts"]
    return e * (1 - (1 - case["sel"] / e) ** case["tok"])


def work(case):
    op, k = case["op"], case["k"]
    if op == "quant":
        n = case["n"] * k
        # x read, blocks written; blocks read, values written
        return {"bytes": n * (SIZE[case["x"]] + 2 * 17 / 32 + SIZE[case["out"]]), "flops": 4.0 * n}
    if op == "rows":
        tok, n, m = case["tok"], case["n"], 2 if case["pair"] else 1
        return {"bytes": m * n * k * 17 / 32 + tok * (k * SIZE[case["x"]] + n * SIZE[case["y"]]),
                "flops": 2.0 * m * tok * n * k}
    kept = case["tok"] * case["sel"] * (1 - case["dropped"])
    if op == "experts":
        n, m = case["n"], 2 if case["pair"] else 1
        xs = case["tok"] if case["gathered"] else kept
        return {"bytes": m * touched(case) * n * k * 17 / 32 + xs * k * SIZE[case["x"]] + kept * n * SIZE[case["y"]],
                "flops": 2.0 * m * kept * n * k}
    x, y, tok, slots = SIZE[case["x"]], SIZE[case["y"]], case["tok"], case["tok"] * case["sel"]
    if case["grad"]:
        # dout and y read, dy written and read again by the gather's gradient, dx written
        return {"bytes": 2 * tok * k * y + 3 * kept * k * x + 12 * slots, "flops": 4.0 * kept * k}
    # ids read, the sort's arrays written; x read, sorted rows written; sorted rows read, sums written
    return {"bytes": 16 * slots + tok * k * (x + y) + 2 * kept * k * x, "flops": 2.0 * kept * k}


# --- the definition in 64 bits ---------------------------------------------------------

def nearest(x, dtype):
    """Quantised and decoded values by search: of the format's values at the block's scale, the nearest (of two
    equally near, the one of even code)."""
    v = x.double().reshape(-1, 32)
    out = torch.empty_like(v)
    grid = torch.tensor(E2M1[:8], dtype=torch.float64, device=v.device)
    for i in range(0, v.shape[0], 1 << 18):
        b = v[i:i + (1 << 18)]
        a = b.abs().amax(1)
        e = torch.floor(torch.log2(a.clamp(min=1e-300)))
        e = e + (torch.exp2(e + 1) <= a).double() - (torch.exp2(e) > a).double()
        scale = torch.exp2(e.sub(2).clamp(-127, 127))[:, None, None]
        off = (b.abs()[..., None] - grid * scale).abs() * (1.0 / scale) + torch.arange(8, device=v.device) % 2 * 1e-9
        got = grid[off.argmin(-1)] * scale[..., 0] * torch.where(torch.signbit(b), -1.0, 1.0)
        out[i:i + (1 << 18)] = torch.where(torch.isfinite(a)[:, None], got, math.nan)
    return out.view(x.shape).to(dtype).double()


def exact(case, seed):
    s = prepare(case, seed)
    op, k = case["op"], case["k"]
    if op == "quant":
        return nearest(s["x"], FLOATS[case["out"]])
    if op in ("rows", "experts"):
        x = values(s["x"], k, torch.float64) if case["x"] == "mxfp4" else s["x"].double()

    def pair_or_one(a, ws):
        out = [a @ values(w, k, torch.float64).T for w in ws]
        return out[0] * torch.sigmoid(out[0]) * out[1] if case["pair"] else out[0]

    if op == "rows":
        return pair_or_one(x, [w[case["skip"]:case["skip"] + case["n"]] for w in s["w"]])
    if op == "experts":
        n, sel, at = case["n"], case["sel"], s["offsets"].tolist()
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            lo, hi = at[e], at[e + 1]
            if hi > lo:
                rows_ = s["slots"][lo:hi].long() // sel if case["gathered"] else slice(lo, hi)
                y[lo:hi] = pair_or_one(x[rows_], [w[e * n:(e + 1) * n] for w in s["w"]])
        return y
    w = s["w"].double()
    if case["grad"]:
        dy = torch.zeros(s["dy"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(w.shape, dtype=torch.float64, device=DEV)
        dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device=DEV)
        dout = s["dout"].double()
        for j in range(case["sel"]):
            kept = s["pos"][:, j] >= 0
            p = s["pos"][kept, j].long()
            dy[p] = (w[kept, j, None] * dout[kept])
            dw[kept, j] = (dout[kept] * s["y"][p].double()).sum(1)
            dx[kept] += dy[p].to(s["dy"].dtype).double()
        return dy, dw, dx
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    flat = s["ids"].flatten().tolist()
    order = [i for _, i in sorted((e, i) for i, e in enumerate(flat) if 0 <= e < case["experts"])]
    xs = torch.zeros(s["xs"].shape, dtype=torch.float64, device=DEV)
    xs[:len(order)] = s["x"][torch.tensor(order, device=DEV) // case["sel"]].double() if order else xs[:0]
    pos = torch.full((len(flat),), -1)
    pos[torch.tensor(order, dtype=torch.long)] = torch.arange(len(order))
    pos = pos.view(s["ids"].shape).to(DEV)
    for j in range(case["sel"]):
        kept = pos[:, j] >= 0
        out[kept] += w[kept, j, None] * s["y"][pos[kept, j]].double()
    return None, None, None, xs, out
