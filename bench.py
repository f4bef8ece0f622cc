"""Benchmark of the batch-1 dequant-GEMV path on one MI355X.

Default workload: the full decode weight pass of a synthetic 20B-class dense
model, Q8_0, 44 layers, hidden 6144, FFN 24576 (per layer QKV 18432x6144,
out 6144x6144, up 24576x6144, down 6144x24576; 21.18 GB resident in HBM).  A
step is one token: the 176 GEMVs of the pass, in order, each fed by the RMS
carry of the previous one (the attention over a single position returns V, so
the carry after QKV is the RMS-normalised V third).  Weights are random-init
synthetic blocks; nothing is cached or skipped between tokens.  Each GEMV is
one qgemv_rows_op launch that normalises its raw input as it loads it (the
up projection stores gelu(u)).  A token's 176 launches are captured once into
a HIP graph that each timed token replays (--eager issues them from the host
instead); --chain runs the pass as one persistent chain launch per token.

Printed: one JSON line with the headline metric (effective weight GB/s of the
whole timed region = weight bytes read / wall time), the roofline of the
dominant kernel (its launches timed with HIP events on the launch stream), the
same run's streaming-read ceiling, the CPU oracle timed on a bounded sample of
the same pass (all permitted threads and one), parity of every GEMV of the first
and last timed token against the oracle (teacher-forced on a bit-identical
replay of the timed tokens) and the oracle's own free-running first token, and
the figures of the other workloads below at their quoted sizes (--no-extras
leaves them out).

Other workloads (--workload): q4_0_4096, moe_mxfp4, ffn_streamed, q8_0_256, and
q4_k_m_dense20b (the same pass with Q4_K QKV/out/up and a Q6_K down
projection, 12.9 GB), dense20b_batch (--batch tokens per step through
qgemv_rows_batch), moe_streamed (the MoE experts streamed from pinned host
memory: ring, plan and zero copy), dense20b_context (the pass with the
attention of its token over --context cached positions in place of the V
third).  ffn_streamed takes --leg to run one of
its ring, plan or zero-copy legs alone.
"""
from __future__ import annotations

import argparse
import ctypes
import json
import os
import platform
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import synth  # noqa: E402

METRIC = "effective weight GB/s (% of HBM peak) of dequant-GEMV; decode tokens/s equiv"
HBM_PEAK_GBS = 8000.0
TOL = 1e-4


def kernel_source_sha256():
    """SHA-256 over every kernel source file, in build order."""
    import hashlib
    from quantized_gemv_gguf_amd import build as qb
    h = hashlib.sha256()
    try:
        for path in qb.source_paths():
            h.update(open(path, "rb").read())
    except OSError:
        return None
    return h.hexdigest()


def profiled_traffic(kernel: str):
    """HBM bytes per launch of `kernel` from a committed rocprofv3 counter
    summary (profiles/*_hbm_traffic.md), if it was taken on the kernel source
    as it is now; else None."""
    import glob
    sha = kernel_source_sha256()
    if sha is None:
        return None
    for path in sorted(glob.glob(os.path.join(ROOT, "profiles", "*_hbm_traffic.md"))):
        vals = {}
        for line in open(path).read().splitlines():
            if "=" in line and not line.startswith(("#", "|", "`")):
                k, v = [t.strip() for t in line.split("=", 1)]
                vals[k] = v
        v = vals.get(f"traffic_bytes_per_launch {kernel}")
        if v and vals.get("kernel_source_sha256") == sha:
            return float(v)
    return None


def threads() -> int:
    """Host threads for the oracle and the generators: every CPU this process
    may run on, capped by OMP_NUM_THREADS where the host sets it (a host
    shared by several GPUs may give each its share of the cores that way)."""
    try:
        n = len(os.sched_getaffinity(0))
    except (AttributeError, OSError):
        n = os.cpu_count() or 1
    cap = int(os.environ.get("OMP_NUM_THREADS", 0) or 0)
    return max(1, min(n, cap) if cap > 0 else n)


def cpu_model() -> str:
    """The CPU's full model string, with its family/model/stepping numbers."""
    info = {}
    try:
        for line in open("/proc/cpuinfo"):
            if ":" in line:
                k, v = [t.strip() for t in line.split(":", 1)]
                info.setdefault(k, v)
    except OSError:
        pass
    name = info.get("model name") or platform.processor() or "unknown"
    extra = ", ".join(f"{k} {info[k]}" for k in ("cpu family", "model", "stepping") if k in info)
    return f"{name} ({extra})" if extra else name


def host_info() -> dict:
    try:
        aff = len(os.sched_getaffinity(0))
    except (AttributeError, OSError):
        aff = None
    return {"cpu_model": cpu_model(), "nproc": os.cpu_count(), "affinity_cpus": aff,
            "omp_num_threads": os.environ.get("OMP_NUM_THREADS")}


def sha256_of(t) -> str:
    """SHA-256 of a tensor's bytes (I4: output hashes compared across runs)."""
    import hashlib
    a = t.detach().contiguous().cpu().numpy()
    return hashlib.sha256(a.tobytes()).hexdigest()


def read_ceiling(dev, nbytes=4 << 30, reps=9):
    """The same run's plain streaming-read rate (qgemv_read_ceiling over 4 GiB,
    far above the 256 MB MALL): median of `reps` reads, HIP events around each."""
    import torch
    import quantized_gemv_gguf_amd as q
    buf = torch.ones(nbytes, dtype=torch.uint8, device=dev)
    sink = torch.zeros(1, dtype=torch.int32, device=dev)
    for _ in range(2):
        q.qgemv_read_ceiling(buf, sink)
    ms = []
    for _ in range(reps):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        q.qgemv_read_ceiling(buf, sink)
        e1.record()
        torch.cuda.synchronize()
        ms.append(e0.elapsed_time(e1))
    med = float(np.median(ms))
    del buf
    torch.cuda.empty_cache()
    gbs = nbytes / (med / 1e3) / 1e9
    return {"GBs": gbs, "pct_hbm_peak": 100.0 * gbs / HBM_PEAK_GBS, "bytes_per_read": nbytes,
            "ms_per_read_median": med, "reads": reps,
            "kernel": "qgemv_read_ceiling: 2048 x 256 lanes, one 16-byte non-temporal load per lane per step"}


# --- the dense decode pass -------------------------------------------------------

class DensePass:
    """Weights, buffers and prepared C-ABI calls of the synthetic dense model."""

    def __init__(self, layers, hidden, ffn, dev, eps=1e-6, verbose=True, cfg=5):
        import torch
        import quantized_gemv_gguf_amd as q
        self.q, self.torch = q, torch
        self.L, self.H, self.F, self.dev, self.eps = layers, hidden, ffn, dev, eps
        self.cfg = cfg
        self.fmts = synth.CONFIGS[cfg]["fmts"]  # format of qkv, out, up, down
        self.shapes = synth.dense_layer_shapes(hidden, ffn)
        self.lib = q.lib()
        self.stream = torch.cuda.current_stream().cuda_stream
        t0 = time.time()
        maxbytes = max(r * synth.row_bytes(f, k) for f, (_, r, k) in zip(self.fmts, self.shapes))
        staging = torch.empty(maxbytes, dtype=torch.uint8, pin_memory=True)
        self.w = []  # [layer][matrix] device tensors
        for l in range(layers):
            row = []
            for m, (_, r, k) in enumerate(self.shapes):
                f = self.fmts[m]
                nbytes = r * synth.row_bytes(f, k)
                view = staging[:nbytes].numpy().reshape(r, synth.row_bytes(f, k))
                synth.blocks(f, r, k, self.seed(l, m), out=view, threads=threads())
                t = torch.empty(nbytes, dtype=torch.uint8, device=dev)
                t.copy_(staging[:nbytes], non_blocking=False)
                row.append(t)
            self.w.append(row)
            if verbose and (l % 11 == 10 or l == layers - 1):
                print(f"[bench] generated {l + 1}/{layers} layers ({time.time() - t0:.1f}s)", file=sys.stderr,
                      flush=True)
        f32 = dict(dtype=torch.float32, device=dev)
        self.qkv = torch.empty(3 * hidden, **f32)
        self.o = torch.empty(hidden, **f32)
        self.u = torch.empty(ffn, **f32)
        self.a = torch.empty(ffn, **f32)
        self.d = torch.empty(hidden, **f32)
        self.c = torch.empty(hidden, **f32)
        self.x0 = torch.from_numpy(synth.x_vec(hidden, synth.seed_of(5, 999))).to(dev)
        # prepared calls: (matrix struct, rows, x ptr, y ptr, bytes, k)
        ins = [self.c, self.c, self.c, self.a]
        outs = [self.qkv, self.o, self.u, self.d]
        self.mats, self.calls = [], []
        for l in range(layers):
            for m, (_, r, k) in enumerate(self.shapes):
                cm = q.qg_matrix(self.w[l][m].data_ptr(), self.fmts[m], 0, r, k, self.w[l][m].numel())
                self.mats.append(cm)
                self.calls.append((ctypes.byref(cm), r, ins[m].data_ptr(), outs[m].data_ptr(),
                                   self.w[l][m].numel(), k, m))
        self.v_ptr = self.qkv.data_ptr() + 4 * 2 * hidden  # the V third of QKV
        self.bytes_per_token = sum(c[4] for c in self.calls)
        # fused launches (qgemv_rows_op): each GEMV normalises its raw input as it
        # loads it; the up projection stores gelu(u).  d carries from token to token.
        fin = [self.d.data_ptr(), self.v_ptr, self.o.data_ptr(), self.a.data_ptr()]
        fout = [self.qkv, self.o, self.a, self.d]
        self.fcalls = []
        for l in range(layers):
            for m, (_, r, k) in enumerate(self.shapes):
                mp, _, _, _, nbytes, _, _ = self.calls[4 * l + m]
                self.fcalls.append((mp, r, fin[m], fout[m].data_ptr(), nbytes, k, m,
                                    q.OUT_GELU if m == 2 else q.OUT_Y))

    def seed(self, layer, m):
        return synth.seed_of(self.cfg, 4 * layer + m)

    def kernel_name(self, m):
        """Name of the GEMV variant matrix m of a layer runs: format and k."""
        return f"gemv_{synth.FMT_NAMES[self.fmts[m]]}_k{self.shapes[m][2]}"

    # -- the pass as one chain: one persistent launch per token --
    def build_chain(self):
        """Steps (l, m) in pass order, each with its own output buffer; the
        carry is fused into the next step's x-load.  The last step writes
        `xin`, which the first step of the next token normalises."""
        torch, q = self.torch, self.q
        H, F = self.H, self.F
        if set(self.fmts) != {q.Q8_0}:
            raise ValueError("chains run the 32-weight formats only")
        f32 = dict(dtype=torch.float32, device=self.dev)
        self.xin = self.x0.clone()
        self.ys = []
        steps = []
        prev = self.xin
        for l in range(self.L):
            outs = [torch.empty(3 * H, **f32), torch.empty(H, **f32), torch.empty(F, **f32),
                    self.xin if l == self.L - 1 else torch.empty(H, **f32)]
            srcs = [prev, outs[0][2 * H:3 * H], outs[1], outs[2]]
            ops = [q.IN_RMS, q.IN_RMS, q.IN_RMS, q.IN_GELU_RMS]
            for m, (_, r, k) in enumerate(self.shapes):
                W = q.Matrix(self.w[l][m], q.Q8_0, r, k)
                steps.append(q.ChainStep([q.ChainWindow(W, 0, r, srcs[m], outs[m])], ops[m], self.eps))
            self.ys.append((outs, srcs, ops))
            prev = outs[3]
        self.chain = q.Chain(q.Q8_0, steps)
        self.chain_handle = ctypes.c_void_p(self.chain.handle)

    def reset_chain(self):
        self.xin.copy_(self.x0)

    def token_chain(self, ev=None):
        if ev is not None:
            ev[0].record()
        rc = self.lib.qgemv_chain_run(self.chain_handle, self.stream)
        if ev is not None:
            ev[1].record()
        if rc != 0:
            raise RuntimeError(f"qgemv_chain_run failed: {rc}")

    def reset(self):
        """c = rms(x0): the carry the first token starts from."""
        rc = self.lib.qgemv_rms_carry(self.x0.data_ptr(), self.c.data_ptr(), self.H, self.eps, 0, self.stream)
        assert rc == 0

    def reset_fused(self):
        self.d.copy_(self.x0)

    def token_fused(self, events=None, hook=None, stream=None, only=None):
        """One token as 176 fused GEMV launches (qgemv_rows_op).  events: one
        (start, end) pair per GEMV, recorded around it on the launch stream;
        only: indices of the launches to issue (timing of one kernel variant)."""
        L, q = self.lib, self.q
        st = self.stream if stream is None else stream
        for i, (mp, r, xp, yp, nbytes, k, m, out_op) in enumerate(self.fcalls):
            if only is not None and i not in only:
                continue
            if events is not None:
                events[i][0].record()
            rc = L.qgemv_rows_op(mp, 0, r, xp, None, q.IN_RMS, self.eps, out_op, yp, 0, st)
            if events is not None:
                events[i][1].record()
            if rc != 0:
                raise RuntimeError(f"qgemv_rows_op failed: {rc}")
            if hook is not None:
                hook(i, m)

    def token(self, events=None, hook=None):
        """One token's pass.  events: list of (start, end) torch events, one
        pair per GEMV, recorded around it on the launch stream."""
        L = self.lib
        H, F, st, eps = self.H, self.F, self.stream, self.eps
        carry = [(self.v_ptr, self.c.data_ptr(), H, 0), (self.o.data_ptr(), self.c.data_ptr(), H, 0),
                 (self.u.data_ptr(), self.a.data_ptr(), F, 1), (self.d.data_ptr(), self.c.data_ptr(), H, 0)]
        for i, (mp, r, xp, yp, nbytes, k, m) in enumerate(self.calls):
            if events is not None:
                events[i][0].record()
            rc = L.qgemv_rows(mp, 0, r, xp, yp, 0, st)
            if events is not None:
                events[i][1].record()
            if rc != 0:
                raise RuntimeError(f"qgemv_rows failed: {rc}")
            if hook is not None:
                hook(i, m)
            vp, op, n, g = carry[m]
            rc = L.qgemv_rms_carry(vp, op, n, eps, g, st)
            if rc != 0:
                raise RuntimeError(f"qgemv_rms_carry failed: {rc}")


FMT_LABEL = {5: "Q8_0", 6: "Q4_K (QKV, out, up) + Q6_K (down)"}


def dense_workload(args, dev, cfg=5):
    import torch
    c = synth.CONFIGS[cfg]
    layers = args.layers or c["layers"]
    model = DensePass(layers, c["hidden"], c["ffn"], dev, cfg=cfg)
    if args.chain:
        return dense_chain_workload(args, dev, model, c, layers)
    torch.cuda.synchronize()
    model.reset_fused()
    for _ in range(args.warmup):
        model.token_fused()
    torch.cuda.synchronize()
    n = len(model.fcalls)
    graph = None
    if not args.eager:
        # one token's 176 launches captured once, replayed per token; the
        # carry is put back afterwards, so the timed tokens start from the
        # same carry (and end on the same bits) as in the eager mode
        d_keep = model.d.clone()
        cap = torch.cuda.Stream()
        cap.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(cap):
            model.token_fused(stream=cap.cuda_stream)
        torch.cuda.current_stream().wait_stream(cap)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=cap):
            model.token_fused(stream=cap.cuda_stream)
        torch.cuda.synchronize()
        for _ in range(max(args.warmup, 1)):
            graph.replay()
        model.d.copy_(d_keep)
        torch.cuda.synchronize()
    # the carry entering the first timed token: the timed tokens are replayed
    # from it afterwards for the parity check (I4: the replay must give the
    # timed run's bits)
    d_start = model.d.clone()
    g0, g1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    g0.record()
    for s in range(args.steps):
        if graph is not None:
            graph.replay()
        else:
            model.token_fused()
    g1.record()
    torch.cuda.synchronize()
    wall = time.perf_counter() - t0
    gpu_ms = g0.elapsed_time(g1)
    d_end = model.d.clone()
    eager = None
    if graph is not None:
        # the same number of tokens issued from the host, right after, for
        # comparison (timing only: the parity replay below starts from d_start)
        torch.cuda.synchronize()
        t0e = time.perf_counter()
        for s in range(args.steps):
            model.token_fused()
        torch.cuda.synchronize()
        we = time.perf_counter() - t0e
        eager = {"value": model.bytes_per_token * args.steps / we / 1e9, "ms_per_step": we / args.steps * 1e3}
    # per-kernel durations: right after the timed region, each kernel variant's
    # launches of two tokens run back to back on the launch stream, bracketed by
    # one pair of HIP events (an event pair around every single launch would
    # add its own packets and gaps to each measured launch)
    per_k = {}
    for kk in sorted({model.kernel_name(c_[6]) for c_ in model.fcalls}):
        sub = [i for i, c_ in enumerate(model.fcalls) if model.kernel_name(c_[6]) == kk]
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(2):
            model.token_fused(only=sub)
        e1.record()
        torch.cuda.synchronize()
        per_k[kk] = [2 * sum(model.fcalls[i][4] for i in sub), e0.elapsed_time(e1), 2 * len(sub)]
    total_bytes = model.bytes_per_token * args.steps
    gbs = total_bytes / wall / 1e9
    kernels = {}
    for k, (b, ms, cnt) in sorted(per_k.items()):
        kernels[k] = {"launches": cnt, "avg_us": ms / cnt * 1e3, "avg_bytes": b / cnt,
                      "GBs": b / (ms / 1e3) / 1e9}
    dom_k = max(per_k, key=lambda k: per_k[k][1])
    b, ms, cnt = per_k[dom_k]
    achieved = b / (ms / 1e3) / 1e9
    res = {
        "value": gbs,
        "ms_per_step": wall / args.steps * 1e3,
        "tokens_per_s": args.steps / wall,
        "pct_hbm_peak": 100.0 * gbs / HBM_PEAK_GBS,
        "gpu_event_ms_per_step": gpu_ms / args.steps,
        "bytes_per_token": model.bytes_per_token,
        "config": {"workload": c["name"], "layers": layers, "hidden": c["hidden"], "ffn": c["ffn"],
                   "format": FMT_LABEL[cfg], "tokens": args.steps, "gemvs_per_token": n,
                   "weight_bytes_per_token": model.bytes_per_token,
                   "launch": "176 fused GEMV launches per token (RMS carry in the x-load, GELU in the store)"
                             + (", one HIP graph per token" if graph is not None else "")},
        "roofline": {"bound": "hbm", "kernel": dom_k, "achieved": achieved,
                     "peak": HBM_PEAK_GBS, "unit": "GB/s", "frac": achieved / HBM_PEAK_GBS,
                     "traffic": profiled_traffic(dom_k), "avg_launch_us": ms / cnt * 1e3,
                     "bytes_per_launch": b / cnt},
        "kernels": kernels,
        "sha256_final_carry": sha256_of(d_end),
    }
    if eager is not None:
        res["eager_launches"] = eager
    # identity: tokens/s = bandwidth / active bytes per token
    assert abs(res["tokens_per_s"] - gbs * 1e9 / model.bytes_per_token) <= 1e-9 * res["tokens_per_s"]
    if not args.no_check:
        res["parity"] = dense_replay_parity(model, layers, d_start, d_end, args.steps,
                                            free_running=not args.no_free_running)
    if not args.no_cpu_baseline:
        res["cpu_baseline"] = dense_cpu_baselines(model, args.cpu_seconds)
    del model
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return res


def dense_replay_parity(model, layers, d_start, d_end, steps, free_running=True):
    """Parity of the timed tokens.  They are replayed from the carry that
    entered the first one; the replay must end on the timed run's bits (I4),
    so checking it checks them.  On the first and the last timed token every
    one of the 176 GEMVs is teacher-forced (dense_parity); the free-running
    oracle (its own fp64 sums from the same starting carry, inputs rounded to
    fp32 per step) is reported for the first token, not gated."""
    import torch
    model.d.copy_(d_start)
    forced = {}
    d_after0 = None
    for t in range(steps):
        if t in (0, steps - 1):
            forced[t] = dense_parity(model, layers, seed=7 + t, every_gemv=True)
        else:
            model.token_fused()
        if t == 0:
            torch.cuda.synchronize()
            d_after0 = model.d.cpu().numpy().astype(np.float64)
    torch.cuda.synchronize()
    same = bool(torch.equal(model.d.view(torch.int32), d_end.view(torch.int32)))
    worst_c = max(v["max_componentwise"] for v in forced.values())
    worst_n = max(v["max_normwise_sampled"] for v in forced.values())
    out = {"teacher_forced": {"tokens": sorted({0, steps - 1}), "gemvs_per_token": len(model.fcalls),
                              "rows_checked": sum(v["rows_checked"] for v in forced.values()),
                              "max_componentwise": worst_c, "max_normwise_sampled": worst_n},
           "replay_bit_identical_to_timed_run": same, "tol": TOL,
           "pass": bool(same and worst_c <= TOL and worst_n <= TOL)}
    if free_running:
        out["free_running_token0"] = dense_free_running(model, d_start.cpu().numpy(), d_after0)
    return out


def dense_free_running(model, d_in, d_gpu):
    """The oracle's own pass of one token from the GPU's starting carry (every
    row of every GEMV, fp64 sums; each step's input rounded to fp32 as the
    oracle takes it): the normwise difference of the final carry from the
    GPU's.  Errors compound over 176 steps, so this is reported, not gated."""
    import oracle
    nth = threads()
    t = time.perf_counter()
    c = oracle.rms_carry(d_in.astype(np.float64), model.eps)
    for l in range(model.L):
        fm = model.fmts
        ws = [synth.blocks(fm[m], r, k, model.seed(l, m), threads=nth) for m, (_, r, k) in enumerate(model.shapes)]
        y, _ = oracle.gemv_rows(fm[0], ws[0], *model.shapes[0][1:], c.astype(np.float32), threads=nth)
        c = oracle.rms_carry(y[2 * model.H:3 * model.H], model.eps)
        y, _ = oracle.gemv_rows(fm[1], ws[1], *model.shapes[1][1:], c.astype(np.float32), threads=nth)
        c = oracle.rms_carry(y, model.eps)
        y, _ = oracle.gemv_rows(fm[2], ws[2], *model.shapes[2][1:], c.astype(np.float32), threads=nth)
        act = oracle.rms_carry(y, model.eps, gelu=True)
        y, _ = oracle.gemv_rows(fm[3], ws[3], *model.shapes[3][1:], act.astype(np.float32), threads=nth)
        c = y  # the raw down output is the carry the next token's first GEMV normalises
    err = np.abs(d_gpu - c)
    return {"max_abs_diff_over_max_abs": float(err.max() / np.abs(c).max()),
            "mean_abs_diff_over_mean_abs": float(err.mean() / np.abs(c).mean()),
            "seconds": round(time.perf_counter() - t, 1), "gated": False}


def dense_chain_workload(args, dev, model, c, layers):
    """The pass as one chain launch per token (qgemv_chain_run)."""
    import torch
    model.build_chain()
    model.reset_chain()
    for _ in range(args.warmup):
        model.token_chain()
    model.chain.check()
    events = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
              for _ in range(args.steps)]
    g0, g1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    g0.record()
    for s in range(args.steps):
        model.token_chain(events[s])
    g1.record()
    torch.cuda.synchronize()
    wall = time.perf_counter() - t0
    model.chain.check()
    gpu_ms = g0.elapsed_time(g1)
    launch_ms = [e0.elapsed_time(e1) for e0, e1 in events]
    avg_ms = sum(launch_ms) / len(launch_ms)
    b = model.bytes_per_token
    gbs = b * args.steps / wall / 1e9
    achieved = b / (avg_ms / 1e3) / 1e9
    kname = "chain_q8_0_dense20b"
    res = {
        "value": gbs,
        "ms_per_step": wall / args.steps * 1e3,
        "tokens_per_s": args.steps / wall,
        "pct_hbm_peak": 100.0 * gbs / HBM_PEAK_GBS,
        "gpu_event_ms_per_step": gpu_ms / args.steps,
        "bytes_per_token": b,
        "config": {"workload": c["name"], "layers": layers, "hidden": c["hidden"], "ffn": c["ffn"],
                   "format": "Q8_0", "tokens": args.steps, "gemvs_per_token": len(model.calls),
                   "weight_bytes_per_token": b, "launch": "one chain launch per token",
                   "grid_workgroups": model.chain.grid},
        "roofline": {"bound": "hbm", "kernel": kname, "achieved": achieved, "peak": HBM_PEAK_GBS,
                     "unit": "GB/s", "frac": achieved / HBM_PEAK_GBS, "traffic": profiled_traffic(kname),
                     "avg_launch_us": avg_ms * 1e3, "bytes_per_launch": b},
        "kernels": {kname: {"launches": args.steps, "avg_us": avg_ms * 1e3, "min_us": min(launch_ms) * 1e3,
                            "max_us": max(launch_ms) * 1e3, "avg_bytes": b, "GBs": achieved}},
    }
    assert abs(res["tokens_per_s"] - gbs * 1e9 / b) <= 1e-9 * res["tokens_per_s"]
    if not args.no_check:
        res["parity"] = dense_chain_parity(model, layers)
    if not args.no_cpu_baseline:
        res["cpu_baseline"] = dense_cpu_baselines(model, args.cpu_seconds)
    model.chain.close()
    torch.cuda.synchronize()
    return res


def dense_chain_parity(model, layers, n_rows=48, seed=7):
    """Teacher-forced check of one more chain token: for every step of layers
    0 and layers-1, the oracle normalises the GPU's own input vector in fp64
    and multiplies sampled rows (weights regenerated on the host)."""
    import torch
    import oracle
    rng = np.random.default_rng(seed)
    x_first = model.xin.clone()
    model.token_chain()
    model.chain.check()
    torch.cuda.synchronize()
    worst_n, worst_c, checked = 0.0, 0.0, 0
    for l in sorted({0, layers - 1}):
        outs, srcs, ops = model.ys[l]
        for m, (_, r, k) in enumerate(model.shapes):
            src = x_first if (l == 0 and m == 0) else srcs[m]
            x = oracle.rms_carry(src.cpu().numpy().astype(np.float64), model.eps, gelu=(m == 3))
            y = outs[m].cpu().numpy().astype(np.float64)
            rows = np.sort(rng.choice(r, n_rows, replace=False))
            ref, a = np.empty(n_rows), np.empty(n_rows)
            for j, row in enumerate(rows):
                wrow = synth.blocks(synth.Q8_0, r, k, model.seed(l, m), r0=int(row), r1=int(row) + 1, threads=1)
                ref[j], a[j] = [v[0] for v in oracle.gemv_rows(oracle.Q8_0, wrow, 1, k, x, threads=1)]
            err = np.abs(y[rows] - ref)
            worst_c = max(worst_c, float(np.max(err / a)))
            worst_n = max(worst_n, float(err.max() / np.abs(ref).max()))
            checked += n_rows
    ok = worst_c <= TOL and worst_n <= TOL
    return {"rows_checked": checked, "max_componentwise": worst_c, "max_normwise_sampled": worst_n,
            "tol": TOL, "pass": bool(ok), "teacher_forced": "fp64 rms of the GPU's own step inputs"}


def dense_parity(model, layers, n_rows=48, seed=7, every_gemv=False):
    """Teacher-forced check of one token's GEMVs (every GEMV, or those of
    layers 0 and layers-1): each one's input is copied back, the oracle
    normalises it in fp64 and multiplies sampled rows (8 runs of n_rows/8
    consecutive rows, so tile edges are crossed) regenerated on the host."""
    import torch
    import oracle
    rng = np.random.default_rng(seed)
    if every_gemv:
        want = set(range(len(model.fcalls)))
    else:
        want = {0, 1, 2, 3, 4 * (layers - 1), 4 * (layers - 1) + 1, 4 * (layers - 1) + 2, 4 * (layers - 1) + 3}
    # fused launches: GEMV i normalises its raw input (oracle: fp64 RMS of
    # the GPU's own input) and the up projection stores gelu(u)
    outs = [model.qkv, model.o, model.a, model.d]
    worst_n, worst_c = 0.0, 0.0
    checked = 0
    H = model.H
    state = {}
    run = max(1, n_rows // 8)

    def raw_input(i, m):
        if m == 0:
            return state["d_in"]
        if m == 1:
            return model.qkv[2 * H:3 * H].cpu().numpy()
        return (model.o if m == 2 else model.a).cpu().numpy()

    def hook(i, m):
        nonlocal worst_n, worst_c, checked
        if i not in want:
            if m == 3:
                torch.cuda.synchronize()
                state["d_in"] = model.d.cpu().numpy()
            return
        torch.cuda.synchronize()
        x = oracle.rms_carry(raw_input(i, m).astype(np.float64), model.eps, gelu=False)
        y = outs[m].cpu().numpy().astype(np.float64)
        if m == 3:
            state["d_in"] = model.d.cpu().numpy()
        _, r, k = model.shapes[m]
        f = model.fmts[m]
        starts = np.sort(rng.choice(r // run, 8, replace=False)) * run
        rows = np.concatenate([np.arange(s0, s0 + run) for s0 in starts])
        ref, a = np.empty(rows.size), np.empty(rows.size)
        for j, s0 in enumerate(starts):
            w = synth.blocks(f, r, k, model.seed(i // 4, m), r0=int(s0), r1=int(s0) + run, threads=1)
            rr, aa = oracle.gemv_rows(f, w, run, k, x, threads=1)
            ref[j * run:(j + 1) * run], a[j * run:(j + 1) * run] = rr, aa
        if m == 2:  # the stored output is gelu(u): compare u's GELU in fp64
            from math import erfc, sqrt
            ref = np.array([0.5 * v * erfc(-v / sqrt(2.0)) for v in ref])
            # |gelu'| <= 1.13 carries u's error through; the fp32 erfc adds a
            # rounding error relative to |gelu(u)|
            a = 1.13 * a + np.abs(ref)
        err = np.abs(y[rows] - ref)
        with np.errstate(invalid="ignore", divide="ignore"):
            c_ = float(np.max(err / a))
            n_ = float(err.max() / np.abs(ref).max())
        # a degenerate sample (all-zero or non-finite rows) fails the check
        worst_c = max(worst_c, c_ if np.isfinite(c_) else np.inf)
        worst_n = max(worst_n, n_ if np.isfinite(n_) else np.inf)
        checked += rows.size

    torch.cuda.synchronize()
    state["d_in"] = model.d.cpu().numpy()
    model.token_fused(hook=hook)
    torch.cuda.synchronize()
    ok = worst_c <= TOL and worst_n <= TOL
    return {"rows_checked": checked, "gemvs_checked": len(want), "max_componentwise": worst_c,
            "max_normwise_sampled": worst_n, "tol": TOL, "pass": bool(ok)}


def dense_cpu_baselines(model, seconds):
    """The oracle on all host threads (the headline baseline) and on one."""
    allt = dense_cpu_baseline(model, seconds)
    one = dense_cpu_baseline(model, max(2.0, seconds / 3), nth=1)
    allt["one_thread"] = {k: one[k] for k in ("value", "unit", "tokens_per_s_equiv", "sample")}
    allt["threads"] = allt["cores"]
    allt["host"] = host_info()
    return allt


def dense_cpu_baseline(model, seconds, nth=None):
    """The oracle (fp64) on the same pass: token after token, layer by layer
    from token 0's carry, until `seconds` of oracle time have run (weight
    regeneration for the oracle is not timed)."""
    import oracle
    t_oracle = 0.0
    nbytes = 0
    nth = threads() if nth is None else nth
    c = oracle.rms_carry(synth.x_vec(model.H, synth.seed_of(5, 999)).astype(np.float64), model.eps)
    layers_done = 0
    tok = 0
    while t_oracle < seconds:
        for l in range(model.L):
            fm = model.fmts
            ws = [synth.blocks(fm[m], r, k, model.seed(l, m), threads=threads())
                  for m, (_, r, k) in enumerate(model.shapes)]
            t = time.perf_counter()
            y, _ = oracle.gemv_rows(fm[0], ws[0], *model.shapes[0][1:], c.astype(np.float32), threads=nth)
            c = oracle.rms_carry(y[2 * model.H:3 * model.H], model.eps)
            y, _ = oracle.gemv_rows(fm[1], ws[1], *model.shapes[1][1:], c.astype(np.float32), threads=nth)
            c = oracle.rms_carry(y, model.eps)
            y, _ = oracle.gemv_rows(fm[2], ws[2], *model.shapes[2][1:], c.astype(np.float32), threads=nth)
            act = oracle.rms_carry(y, model.eps, gelu=True)
            y, _ = oracle.gemv_rows(fm[3], ws[3], *model.shapes[3][1:], act.astype(np.float32), threads=nth)
            c = oracle.rms_carry(y, model.eps)
            t_oracle += time.perf_counter() - t
            nbytes += sum(w.nbytes for w in ws)
            layers_done += 1
            if t_oracle >= seconds:
                break
        tok += 1
    gbs = nbytes / t_oracle / 1e9
    return {"value": gbs, "unit": "GB/s", "cores": nth, "kind": "oracle",
            "tokens_per_s_equiv": gbs * 1e9 / model.bytes_per_token,
            "sample": f"{layers_done} layer passes ({4 * layers_done} GEMVs, {nbytes / 1e9:.2f} GB of "
                      f"{FMT_LABEL[model.cfg]} weights, {tok} token(s) of the same {model.L}-layer pass), "
                      f"fp64 scalar C oracle, "
                      f"{nth} threads, {t_oracle:.1f} s",
            "cpu": cpu_model()}



# --- other workloads -------------------------------------------------------------------

def _timed(fn, n, torch):
    """(wall seconds, gpu ms) of n calls of fn() on the current stream."""
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    e0.record()
    for i in range(n):
        fn(i)
    e1.record()
    torch.cuda.synchronize()
    return time.perf_counter() - t0, e0.elapsed_time(e1)


def q4_0_workload(args, dev):
    """Q4_0 4096x4096.  A single 9.4 MB matrix sits in the 256 MB MALL when
    re-run, so the timed launches rotate over 128 distinct copies (1.21 GB);
    also timed: one grid over 16 distinct matrices (151 MB) per launch, and
    block_rows 0 vs 512 (bit-identical outputs)."""
    import torch
    import quantized_gemv_gguf_amd as q
    c = synth.CONFIGS[2]
    rows, k = c["rows"], c["k"]
    nbytes = q.qgemv_weight_bytes(q.Q4_0, rows, k)
    ncopy = 128
    base = synth.blocks(q.Q4_0, rows, k, synth.seed_of(2, 0))
    mats = [torch.from_numpy(base).to(dev) for _ in range(ncopy)]
    x = torch.from_numpy(synth.x_vec(k, synth.seed_of(2, 9))).to(dev)
    ys = torch.empty((16, rows), dtype=torch.float32, device=dev)
    L = q.lib()
    st = torch.cuda.current_stream().cuda_stream
    cm = [q.qg_matrix(m.data_ptr(), q.Q4_0, 0, rows, k, nbytes) for m in mats]
    # arguments marshalled once (a tensor view per call costs the host a few µs)
    cmr = [ctypes.byref(m) for m in cm]
    xp, y0p = x.data_ptr(), ys[0].data_ptr()

    def one(i, B=0):
        rc = L.qgemv_rows(cmr[i % ncopy], 0, rows, xp, y0p, B, st)
        assert rc == 0

    arrs = []
    for g in range(ncopy // 16):
        ws = [q.Window(q.Matrix(mats[16 * g + j], q.Q4_0, rows, k), 0, rows, x, ys[j]) for j in range(16)]
        arrs.append((q.qg_window * 16)(*[w.c() for w in ws]))

    def grid(i):
        rc = L.qgemv_windows(q.Q4_0, k, arrs[i % len(arrs)], 16, 0, st)
        assert rc == 0

    for i in range(max(args.warmup, 16)):
        one(i)
    for i in range(max(args.warmup, 2)):
        grid(i)
    n = max(args.steps, 64)
    # the single-matrix launches (about 6 us each) are timed over twice as many
    # launches, so that the stream's start-up is a small part of the figure
    wall1, ms1 = _timed(one, 2 * n, torch)
    wall16, ms16 = _timed(grid, n, torch)
    # the same grid kept busy for longer: after about a millisecond of these
    # launches back to back the device lowers its clocks (the rate recovers
    # when the launches are paced), so the last 128 of 384 are reported apart
    ms16s = None
    if not args.no_sustained:
        _timed(grid, 256, torch)
        _, ms16s = _timed(grid, 128, torch)
    y0 = torch.empty(rows, device=dev)
    y512 = torch.empty(rows, device=dev)
    L.qgemv_rows(ctypes.byref(cm[0]), 0, rows, x.data_ptr(), y0.data_ptr(), 0, st)
    L.qgemv_rows(ctypes.byref(cm[0]), 0, rows, x.data_ptr(), y512.data_ptr(), 512, st)
    torch.cuda.synchronize()
    same = bool(torch.equal(y0.view(torch.int32), y512.view(torch.int32)))
    res = {
        "value": nbytes * 16 * n / (ms16 / 1e3) / 1e9,
        "ms_per_step": ms16 / n,
        "pct_hbm_peak": 100.0 * nbytes * 16 * n / (ms16 / 1e3) / 1e9 / HBM_PEAK_GBS,
        "sha256_y": {"block_rows_0": sha256_of(y0), "block_rows_512": sha256_of(y512)},
        "config": {"workload": c["name"], "format": "Q4_0", "rows": rows, "k": k,
                   "launch": "one grid over 16 distinct matrices (151 MB), rotated over 128 copies"},
        "sustained": None if ms16s is None else {
            "GBs": nbytes * 16 * 128 / (ms16s / 1e3) / 1e9, "us_per_grid": ms16s / 128 * 1e3,
            "note": "the last 128 of 384 grids launched back to back (device clocks lowered by then)"},
        "single_matrix": {"us_per_launch": ms1 / (2 * n) * 1e3, "GBs": nbytes * 2 * n / (ms1 / 1e3) / 1e9,
                          "note": "one 9.4 MB matrix per launch, rotated over 128 copies"},
        "block_rows_0_vs_512_bit_identical": same,
    }
    if not args.no_check:
        import oracle
        ref, a = oracle.gemv_rows(oracle.Q4_0, base, rows, k, x.cpu().numpy())
        err = np.abs(y0.cpu().numpy().astype(np.float64) - ref)
        res["parity"] = {"max_componentwise": float(np.max(err / a)),
                         "max_normwise": float(err.max() / np.abs(ref).max()), "tol": TOL,
                         "pass": bool(np.all(err <= TOL * a) and err.max() <= TOL * np.abs(ref).max())}
    return res


def moe_workload(args, dev):
    """MXFP4 MoE expert GEMV: stacked (128, 2880, 2880) gate/up/down, 4 of 128
    experts per token (seeded uniform top-4), 64 tokens.  Per token: one grid
    over the selected experts' gate and up rows in pairs, storing
    silu(gate) * up (qgemv_expert_swiglu), one grid over the 4 down windows,
    and the router-weighted combine of the 4 expert outputs (seeded weights).
    (SiLU*up fused into the down grid's x-load instead, qgemv_expert_windows_op,
    is slower here: every one of the ~1,400 teams of that small grid evaluates
    it for its whole input slice.)"""
    import torch
    import quantized_gemv_gguf_amd as q
    c = synth.CONFIGS[4]
    E, out, k, ns = c["n_expert"], c["out"], c["k"], c["n_sel"]
    rows = E * out
    host = [synth.blocks(q.MXFP4, rows, k, synth.seed_of(4, t)) for t in range(3)]
    mats = [q.Matrix(torch.from_numpy(h).to(dev), q.MXFP4, rows, k) for h in host]
    ids = synth.expert_ids(E, ns, c["tokens"], synth.seed_of(4, 8))
    xs = torch.from_numpy(np.stack([synth.x_vec(k, synth.seed_of(4, 100 + t)) for t in range(c["tokens"])])).to(dev)
    h = torch.empty(ns * out, dtype=torch.float32, device=dev)
    ye = torch.empty(ns * out, dtype=torch.float32, device=dev)
    y = torch.empty((c["tokens"], out), dtype=torch.float32, device=dev)
    wts = torch.from_numpy(synth.router_weights(c["tokens"], ns, synth.seed_of(4, 9))).to(dev)
    L = q.lib()
    st = torch.cuda.current_stream().cuda_stream
    m1 = (q.qg_matrix * 1)(mats[2].c())
    gate_c, up_c = mats[0].c(), mats[1].c()
    gate_m, up_m = ctypes.byref(gate_c), ctypes.byref(up_c)
    idarr = [(ctypes.c_int32 * ns)(*[int(v) for v in ids[t]]) for t in range(c["tokens"])]
    # device addresses taken once: a tensor view per call costs the host a few
    # µs, which is marshalling, not the path
    xp = [xs[t].data_ptr() for t in range(c["tokens"])]
    wp = [wts[t].data_ptr() for t in range(c["tokens"])]
    yp = [y[t].data_ptr() for t in range(c["tokens"])]
    hp, yep = h.data_ptr(), ye.data_ptr()
    B = args.block_rows

    def token(t):
        t = t % c["tokens"]
        rc = L.qgemv_expert_swiglu(gate_m, up_m, E, idarr[t], ns, xp[t], 0, q.IN_X, 0.0, hp, B, st)
        rc |= L.qgemv_expert_windows(m1, 1, E, idarr[t], ns, hp, out, yep, B, st)
        rc |= L.qgemv_combine(yep, out, ns, wp[t], out, yp[t], st)
        assert rc == 0

    for t in range(args.warmup):
        token(t)
    n = args.steps if args.steps > 0 else c["tokens"]
    wall, ms = _timed(token, n, torch)
    per_tok = 3 * ns * q.qgemv_weight_bytes(q.MXFP4, out, k)
    gbs = per_tok * n / wall / 1e9
    # every token once more at each of the config's block sizes: the outputs
    # must not depend on it (I1); their hashes are recorded (I4)
    hashes, outs = {}, {}
    for Bv in synth.CONFIGS[4]["block_rows"]:
        B = Bv
        for t in range(c["tokens"]):
            token(t)
        torch.cuda.synchronize()
        outs[Bv] = y.clone()
        hashes[f"block_rows_{Bv}"] = sha256_of(y)
    B = args.block_rows
    ref = outs[synth.CONFIGS[4]["block_rows"][0]]
    same = all(bool(torch.equal(o.view(torch.int32), ref.view(torch.int32))) for o in outs.values())
    return {"value": gbs, "ms_per_step": wall / n * 1e3, "tokens_per_s": n / wall,
            "us_per_token": wall / n * 1e6, "pct_hbm_peak": 100.0 * gbs / HBM_PEAK_GBS,
            "bytes_per_token": per_tok, "block_rows_bit_identical": same, "sha256_y_all_tokens": hashes,
            "config": {"workload": c["name"], "format": "MXFP4", "n_expert": E, "out": out, "k": k,
                       "experts_per_token": ns, "tokens": n, "block_rows": args.block_rows,
                       "launches_per_token": "gate/up pair grid storing SiLU*up, down grid, combine",
                       "resident_bytes": 3 * q.qgemv_weight_bytes(q.MXFP4, rows, k)}}


def ffn_streamed_workload(args, dev):
    """Q8_0 FFN trio (gate/up 11008x4096, down 4096x11008) streamed from pinned
    host memory through a lookahead-2 ring at block_rows 128/512/2048; the
    host link is measured in the same run with one 256 MiB pinned H2D copy and
    with copies of each block size.  Outputs are compared bit for bit with the
    resident run."""
    import torch
    import quantized_gemv_gguf_amd as q
    c = synth.CONFIGS[3]
    H, F = c["hidden"], c["ffn"]
    gate = synth.blocks(q.Q8_0, F, H, synth.seed_of(3, 0))
    up = synth.blocks(q.Q8_0, F, H, synth.seed_of(3, 1))
    down = synth.blocks(q.Q8_0, H, F, synth.seed_of(3, 2))

    def pinned(a):
        t = torch.empty(a.shape, dtype=torch.uint8, pin_memory=True)
        t.numpy()[...] = a
        return t

    pin = [pinned(a) for a in (gate, up, down)]
    res_w = [torch.from_numpy(a).to(dev) for a in (gate, up, down)]
    x = torch.from_numpy(synth.x_vec(H, synth.seed_of(3, 9))).to(dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g, u, hh, y = torch.empty(F, **f32), torch.empty(F, **f32), torch.empty(F, **f32), torch.empty(H, **f32)
    per_tok = sum(a.nbytes for a in (gate, up, down))

    def run(ws, streamer=None, B=0, mapped=False):
        W = [q.Matrix(ws[0], q.Q8_0, F, H), q.Matrix(ws[1], q.Q8_0, F, H), q.Matrix(ws[2], q.Q8_0, H, F)]
        if mapped:
            q.qgemv_mapped_windows([q.Window(W[0], 0, F, x, g), q.Window(W[1], 0, F, x, u)])
            q.qgemv_silu_mul(g, u, hh)
            q.qgemv_mapped_rows(W[2], 0, H, hh, y)
        elif streamer is None:
            q.qgemv_windows([q.Window(W[0], 0, F, x, g), q.Window(W[1], 0, F, x, u)])
            q.qgemv_silu_mul(g, u, hh)
            q.qgemv_rows(W[2], 0, H, hh, y)
        else:
            streamer.windows([q.Window(W[0], 0, F, x, g), q.Window(W[1], 0, F, x, u)], B)
            q.qgemv_silu_mul(g, u, hh)
            streamer.rows(W[2], 0, H, hh, y, B)

    run(res_w)
    torch.cuda.synchronize()
    ref = y.clone()
    # resident, for reference: the separate first phase (gate/up grid, SiLU*up)
    # against the SwiGLU pair grid (qgemv_rows_swiglu), each then down
    Wr = [q.Matrix(res_w[0], q.Q8_0, F, H), q.Matrix(res_w[1], q.Q8_0, F, H), q.Matrix(res_w[2], q.Q8_0, H, F)]

    def fused(i=0):
        q.qgemv_rows_swiglu(Wr[0], Wr[1], 0, F, x, hh)
        q.qgemv_rows(Wr[2], 0, H, hh, y)

    resident = {}
    for name, fn in (("separate", lambda i: run(res_w)), ("swiglu_pair", fused)):
        for _ in range(max(args.warmup, 2)):
            fn(0)
        wall_r, _ = _timed(fn, 64, torch)
        resident[name] = {"us_per_token": wall_r / 64 * 1e6, "GBs": per_tok * 64 / wall_r / 1e9,
                          "bit_identical": bool(torch.equal(y.view(torch.int32), ref.view(torch.int32)))}
    # host link: one 256 MiB pinned copy, and copies of each block size
    big = torch.empty(256 << 20, dtype=torch.uint8, pin_memory=True)
    dbig = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
    for _ in range(2):
        dbig.copy_(big, non_blocking=True)
    wall, ms = _timed(lambda i: dbig.copy_(big, non_blocking=True), 5, torch)
    link_256 = (256 << 20) * 5 / (ms / 1e3) / 1e9
    out = {}
    rb_down = q.qgemv_weight_bytes(q.Q8_0, 1, F)
    sizes = (args.block_rows,) if args.block_rows > 0 else (128, 512, 2048)
    leg = getattr(args, "leg", "all")
    for B in sizes:
        blk = B * rb_down
        wall_c, ms_c = _timed(lambda i: dbig[:blk].copy_(big[:blk], non_blocking=True), 64, torch)
        out[str(B)] = {"copy_GBs_at_block_size": blk * 64 / (ms_c / 1e3) / 1e9}
        if leg not in ("all", "ring"):
            continue
        with q.Streamer(B * rb_down, c["lookahead"]) as stv:
            for _ in range(max(args.warmup, 1)):
                run(pin, stv, B)
            torch.cuda.synchronize()
            n = max(args.steps, 8)
            wall_s, ms_s = _timed(lambda i: run(pin, stv, B), n, torch)
            same = bool(torch.equal(y.view(torch.int32), ref.view(torch.int32)))
            link = per_tok * n / wall_s / 1e9
            out[str(B)].update({"link_GBs": link, "ms_per_token": wall_s / n * 1e3,
                                "pct_of_256MiB_copy": 100 * link / link_256,
                                "bit_identical_to_resident": same, "ring_bytes": stv.ring_bytes,
                                "sha256_y": sha256_of(y)})
    # the same walk as a streamed plan (one graph per token: no per-block host work)
    P = [q.Matrix(pin[0], q.Q8_0, F, H), q.Matrix(pin[1], q.Q8_0, F, H), q.Matrix(pin[2], q.Q8_0, H, F)]
    for B in sizes if leg in ("all", "plan") else ():
        steps = [q.PlanGemv([q.Window(P[0], 0, F, x, g), q.Window(P[1], 0, F, x, u)], B),
                 q.PlanSiluMul(g, u, hh), q.PlanGemv([q.Window(P[2], 0, H, hh, y)], B)]
        with q.StreamPlan(B * rb_down, c["lookahead"], steps) as plan:
            for _ in range(max(args.warmup, 1)):
                plan.run()
            torch.cuda.synchronize()
            n = max(args.steps, 8)
            wall_p, _ = _timed(lambda i: plan.run(), n, torch)
            same = bool(torch.equal(y.view(torch.int32), ref.view(torch.int32)))
            link = per_tok * n / wall_p / 1e9
            out[str(B)]["plan"] = {"link_GBs": link, "ms_per_token": wall_p / n * 1e3,
                                   "pct_of_256MiB_copy": 100 * link / link_256, "bit_identical_to_resident": same,
                                   "ring_bytes": plan.ring_bytes}
    cands = [(r.get(kind, r if kind == "ring" else {}).get("link_GBs", 0.0), B, kind)
             for B, r in out.items() for kind in ("ring", "plan")]
    best_rate, best, best_kind = max(cands)
    mapped = None
    if leg in ("all", "mapped"):
        # zero copy: the kernels read the pinned host weights in place over the link
        for _ in range(max(args.warmup, 1)):
            run(pin, mapped=True)
        torch.cuda.synchronize()
        n = max(args.steps, 8)
        wall_m, ms_m = _timed(lambda i: run(pin, mapped=True), n, torch)
        link_m = per_tok * n / wall_m / 1e9
        mapped = {"link_GBs": link_m, "ms_per_token": wall_m / n * 1e3,
                  "pct_of_256MiB_copy": 100 * link_m / link_256,
                  "bit_identical_to_resident": bool(torch.equal(y.view(torch.int32), ref.view(torch.int32)))}
        if best_rate == 0.0:
            best_rate, best, best_kind = link_m, "0", "mapped"
    return {"value": best_rate, "ms_per_step": per_tok / best_rate / 1e6 if best_rate else 0.0, "unit_note":
            "host-link GB/s of the streamed pass (weight bytes copied / wall time)",
            "pct_of_256MiB_copy": 100 * best_rate / link_256, "best_mode": best_kind,
            "bytes_per_token": per_tok, "h2d_256MiB_GBs": link_256, "block_rows": out, "mapped": mapped,
            "resident": resident, "sha256_y_resident": sha256_of(ref),
            "config": {"workload": c["name"], "format": "Q8_0", "hidden": H, "ffn": F,
                       "lookahead": c["lookahead"], "best_block_rows": int(best), "leg": leg}}


def moe_streamed_workload(args, dev):
    """The MXFP4 MoE workload with the expert tensors in pinned host memory
    (the pages' setting: experts that do not fit the GPU are streamed): per
    token the 8 gate/up windows of the 4 selected experts and then their 4
    down windows go through the block ring (lookahead 1, i.e. two slots, and
    lookahead 2) at block_rows 128, 512 and 2880 (whole experts), with SiLU*up
    between; and the same token with the kernels reading the pinned experts
    in place (mapped).
    Rate = selected-expert bytes / wall time, against one 256 MiB pinned copy;
    outputs compared bit for bit with the resident token."""
    import torch
    import quantized_gemv_gguf_amd as q
    c = synth.CONFIGS[4]
    E, out, k, ns = c["n_expert"], c["out"], c["k"], c["n_sel"]
    rows = E * out
    f32 = dict(dtype=torch.float32, device=dev)

    def pinned(a):
        t = torch.empty(a.shape, dtype=torch.uint8, pin_memory=True)
        t.numpy()[...] = a
        return t

    host = [synth.blocks(q.MXFP4, rows, k, synth.seed_of(4, t)) for t in range(3)]
    pin = [pinned(h) for h in host]
    res = [torch.from_numpy(h).to(dev) for h in host]
    del host
    ids = synth.expert_ids(E, ns, c["tokens"], synth.seed_of(4, 8))
    xs = torch.from_numpy(np.stack([synth.x_vec(k, synth.seed_of(4, 100 + t)) for t in range(c["tokens"])])).to(dev)
    gu, h, ye = torch.empty(2 * ns * out, **f32), torch.empty(ns * out, **f32), torch.empty(ns * out, **f32)
    per_tok = 3 * ns * q.qgemv_weight_bytes(q.MXFP4, out, k)

    def token(ws, t, streamer=None, B=0, mapped=False):
        t = t % c["tokens"]
        M = [q.Matrix(w, q.MXFP4, rows, k) for w in ws]
        sel = [int(v) for v in ids[t]]
        gw = [q.Window(M[m], e * out, (e + 1) * out, xs[t], gu[(m * ns + s) * out:(m * ns + s + 1) * out])
              for m in range(2) for s, e in enumerate(sel)]
        dw = [q.Window(M[2], e * out, (e + 1) * out, h[s * out:(s + 1) * out], ye[s * out:(s + 1) * out])
              for s, e in enumerate(sel)]
        if mapped:
            q.qgemv_mapped_windows(gw)
            q.qgemv_silu_mul(gu[:ns * out], gu[ns * out:], h)
            q.qgemv_mapped_windows(dw)
        elif streamer is None:
            q.qgemv_windows(gw)
            q.qgemv_silu_mul(gu[:ns * out], gu[ns * out:], h)
            q.qgemv_windows(dw)
        else:
            streamer.windows(gw, B)
            q.qgemv_silu_mul(gu[:ns * out], gu[ns * out:], h)
            streamer.windows(dw, B)

    n = max(args.steps, 16)
    refs = []
    for t in range(n):
        token(res, t)
        refs.append(ye.clone())
    torch.cuda.synchronize()
    big = torch.empty(256 << 20, dtype=torch.uint8, pin_memory=True)
    dbig = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
    for _ in range(2):
        dbig.copy_(big, non_blocking=True)
    _, ms = _timed(lambda i: dbig.copy_(big, non_blocking=True), 5, torch)
    link_256 = (256 << 20) * 5 / (ms / 1e3) / 1e9
    rb = q.qgemv_weight_bytes(q.MXFP4, 1, k)
    legs = {}

    def measure(name, **kw):
        for t in range(max(args.warmup, 1)):
            token(pin, t, **kw)
        torch.cuda.synchronize()
        same = True
        wall, _ = _timed(lambda i: token(pin, i, **kw), n, torch)
        # bit identity on the last token, against the resident one
        same = bool(torch.equal(ye.view(torch.int32), refs[(n - 1) % len(refs)].view(torch.int32)))
        link = per_tok * n / wall / 1e9
        legs[name] = {"link_GBs": link, "us_per_token": wall / n * 1e6, "pct_of_256MiB_copy": 100 * link / link_256,
                      "bit_identical_to_resident": same}

    for B in (128, 512, out):
        for la in (1, 2):
            with q.Streamer(B * rb, la) as st:
                measure(f"ring_B{B}_lookahead{la}", streamer=st, B=B)
                legs[f"ring_B{B}_lookahead{la}"]["ring_bytes"] = st.ring_bytes
    measure("mapped", mapped=True)
    # streamed plans: one graph per token, re-pointed at the token's experts
    x = torch.empty(k, **f32)
    sel0 = [int(e) for e in ids[0]]
    Pm = [q.Matrix(w, q.MXFP4, rows, k) for w in pin]
    gw = [q.Window(Pm[m], e * out, (e + 1) * out, x, gu[(m * ns + s) * out:(m * ns + s + 1) * out])
          for m in range(2) for s, e in enumerate(sel0)]
    dw = [q.Window(Pm[2], e * out, (e + 1) * out, h[s * out:(s + 1) * out], ye[s * out:(s + 1) * out])
          for s, e in enumerate(sel0)]
    for B, la in ((128, 1), (512, 1), (512, 2), (out, 2)):
        steps = [q.PlanGemv(gw, B), q.PlanSiluMul(gu[:ns * out], gu[ns * out:], h), q.PlanGemv(dw, B)]
        with q.StreamPlan(B * rb, la, steps) as plan:
            def ptoken(t):
                t = t % c["tokens"]
                for s_, e in enumerate(ids[t]):
                    for m in range(3):
                        plan.set_rows(m * ns + s_, int(e) * out)
                x.copy_(xs[t])
                plan.run()
            for t in range(max(args.warmup, 1)):
                ptoken(t)
            torch.cuda.synchronize()
            wall, _ = _timed(ptoken, n, torch)
            same = bool(torch.equal(ye.view(torch.int32), refs[(n - 1) % len(refs)].view(torch.int32)))
            link = per_tok * n / wall / 1e9
            legs[f"plan_B{B}_lookahead{la}"] = {"link_GBs": link, "us_per_token": wall / n * 1e6,
                                                "pct_of_256MiB_copy": 100 * link / link_256,
                                                "bit_identical_to_resident": same, "ring_bytes": plan.ring_bytes}
    best = max(legs, key=lambda kk: legs[kk]["link_GBs"])
    return {"value": legs[best]["link_GBs"], "ms_per_step": legs[best]["us_per_token"] / 1e3,
            "unit_note": "host-link GB/s of the selected experts' bytes per token (bytes / wall time)",
            "bytes_per_token": per_tok, "h2d_256MiB_GBs": link_256, "legs": legs,
            "config": {"workload": c["name"] + "_streamed", "format": "MXFP4", "n_expert": E, "out": out, "k": k,
                       "experts_per_token": ns, "tokens": n, "best": best}}


def q8_0_small_workload(args, dev):
    """Q8_0 256x1024: a launch-latency case (278 KB of weights)."""
    import torch
    import quantized_gemv_gguf_amd as q
    c = synth.CONFIGS[1]
    rows, k = c["rows"], c["k"]
    w = torch.from_numpy(synth.blocks(q.Q8_0, rows, k, synth.seed_of(1, 0))).to(dev)
    x = torch.from_numpy(synth.x_vec(k, synth.seed_of(1, 9))).to(dev)
    y = torch.empty(rows, device=dev)
    L = q.lib()
    st = torch.cuda.current_stream().cuda_stream
    m = q.Matrix(w, q.Q8_0, rows, k).c()
    mr, xp, yp = ctypes.byref(m), x.data_ptr(), y.data_ptr()

    def one(i):
        assert L.qgemv_rows(mr, 0, rows, xp, yp, 0, st) == 0

    for i in range(10):
        one(i)
    n = max(args.steps, 200)
    wall, ms = _timed(one, n, torch)
    nbytes = w.numel()
    res = {"value": nbytes * n / (ms / 1e3) / 1e9, "ms_per_step": ms / n, "sha256_y": sha256_of(y),
           "config": {"workload": c["name"], "format": "Q8_0", "rows": rows, "k": k,
                      "note": "weights stay in cache across launches; a latency figure, not an HBM one"}}
    if not args.no_check:
        import oracle
        ref, a = oracle.gemv_rows(oracle.Q8_0, w.cpu().numpy(), rows, k, x.cpu().numpy())
        err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
        res["parity"] = {"max_componentwise": float(np.max(err / a)),
                         "max_normwise": float(err.max() / np.abs(ref).max()), "tol": TOL,
                         "pass": bool(np.all(err <= TOL * a) and err.max() <= TOL * np.abs(ref).max())}
    return res


def dense_batch_workload(args, dev):
    """The dense 20B-class pass (Q8_0, or --kquant for the Q4_K_M mix) with
    --batch tokens per step: every GEMV a qgemv_rows_batch call on that many
    fixed activation vectors (no carries between GEMVs: a batch of decode
    streams each has its own).  Reported: tokens/s and the weight bytes the
    passes read per step (a pass reads the matrix once for up to four tokens)."""
    import torch
    import quantized_gemv_gguf_amd as q
    import oracle
    cfg = 6 if args.kquant else 5
    c = synth.CONFIGS[cfg]
    layers = args.layers or c["layers"]
    B = args.batch
    mfma = args.mfma
    model = DensePass(layers, c["hidden"], c["ffn"], dev, cfg=cfg)
    H, F = c["hidden"], c["ffn"]
    X = {k: torch.from_numpy(np.stack([synth.x_vec(k, synth.seed_of(10, 1000 * (k // 1024) + t))
                                        for t in range(B)])).to(dev) for k in (H, F)}
    Y = [torch.empty((B, r), dtype=torch.float32, device=dev) for _, r, _ in model.shapes]
    L, st = model.lib, model.stream
    call = "qgemv_rows_mfma" if mfma else "qgemv_rows_batch"

    def passes(k):
        """Tokens per pass for this k (the library's choice, restated for the byte count)."""
        if mfma:
            return [min(16, B - t) for t in range(0, B, 16)]
        nb = k // 32
        wt1 = -(-nb // 64)
        c_ = 1 if (wt1 <= 12 and model.fmts[0] != q.Q4_0) else 2
        out, left = [], B
        while left > 0:
            wt = -(-nb // (64 * c_))
            nt = 4 if left >= 4 and c_ == 1 and wt <= 8 else 2 if left >= 2 and (c_ == 1 or wt <= 8) else 1
            out.append(nt)
            left -= nt
        return out

    def step(_=0):
        for i, (mp, r, _, _, nbytes, k, m) in enumerate(model.calls):
            if mfma:
                rc = L.qgemv_rows_mfma(mp, 0, r, X[k].data_ptr(), k, B, Y[m].data_ptr(), r, st)
            else:
                rc = L.qgemv_rows_batch(mp, 0, r, X[k].data_ptr(), k, B, Y[m].data_ptr(), r, 0, st)
            if rc != 0:
                raise RuntimeError(f"{call} failed: {rc}")

    for _ in range(args.warmup):
        step()
    wall, gpu_ms = _timed(step, args.steps, torch)
    per_step_read = sum(len(passes(k)) * nbytes for (_, r, _, _, nbytes, k, m) in model.calls)
    tok_bytes = model.bytes_per_token * B
    # parity: sampled rows of the first layer's four GEMVs, every token
    worst = 0.0
    rng = np.random.default_rng(3)
    step()
    torch.cuda.synchronize()
    for m, (_, r, k) in enumerate(model.shapes):
        y = Y[m].cpu().numpy()  # the last layer's outputs
        rows = np.sort(rng.choice(r, 16, replace=False))
        for row in rows:
            wrow = synth.blocks(model.fmts[m], r, k, model.seed(layers - 1, m), r0=int(row), r1=int(row) + 1,
                                threads=1)
            for t in range(B):
                ref, a = oracle.gemv_rows(model.fmts[m], wrow, 1, k, X[k][t].cpu().numpy(), threads=1)
                worst = max(worst, float(abs(y[t, row] - ref[0]) / a[0]) if a[0] > 0 else np.inf)
    return {"value": per_step_read * args.steps / wall / 1e9, "ms_per_step": wall / args.steps * 1e3,
            "tokens_per_s": B * args.steps / wall, "token_equiv_GBs": tok_bytes * args.steps / wall / 1e9,
            "bytes_read_per_step": per_step_read, "weight_bytes_per_token": model.bytes_per_token,
            "config": {"workload": c["name"] + f"_batch{B}" + ("_mfma" if mfma else ""), "layers": layers,
                       "format": FMT_LABEL[cfg], "tokens_per_step": B,
                       "passes_per_gemv": {str(k): passes(k) for k in (H, F)},
                       "launch": f"176 {call} calls per step"},
            "parity": {"rows_checked": 16 * 4 * B, "max_componentwise": worst, "tol": TOL,
                       "pass": bool(worst <= TOL)}}


def dense_context_workload(args, dev):
    """The dense 20B-class pass with attention over a paged fp16 cache: 64 heads
    of 96, a quarter of each turned by its position, --context positions of
    synthetic keys and values.  The prompt's sequence is forked, and the fork
    decodes: a token makes room in the pool (the first copies the shared last
    page), and between a layer's QKV and output products come qgemv_kv_append
    and qgemv_kv_attend.  A token is one HIP graph (--eager: issued from the
    host).  The rate counts weight bytes only, as the pass without attention
    does; the cache's are reported beside it."""
    import torch
    import quantized_gemv_gguf_amd as q
    c = synth.CONFIGS[5]
    layers = args.layers or c["layers"]
    H, heads, rot, size = c["hidden"], 64, 24, 16
    dim, n0 = H // heads, args.context
    if n0 < 1:
        raise SystemExit("bench.py: --context must be at least 1")
    model = DensePass(layers, H, c["ffn"], dev)
    total = n0 + args.warmup + args.steps + 2  # (and what is run before a capture)
    wide = -(-total // size)
    pages = 2 * wide
    i32 = dict(dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(synth.seed_of(5, 500))
    cache = q.KvCache(*(torch.randn(layers, pages, heads, size, dim, generator=g, dtype=torch.float16, device=dev)
                        for _ in range(2)))
    pool = q.KvPool(torch.full((2, wide), -1, **i32), torch.zeros(2, **i32), torch.zeros(pages, **i32),
                    torch.zeros(-(-pages // 32), **i32), size,
                    torch.empty(q.qgemv_kv_pool_bytes(2, wide, pages), dtype=torch.uint8, device=dev))
    q.qgemv_kv_resize(pool, cache, torch.tensor([n0, -1], **i32))
    q.qgemv_kv_fork(pool, torch.tensor([0, 0], **i32))
    freqs, mscale = q.qgemv_rope_freqs(rot)
    rope = q.Rope(torch.tensor(freqs, dtype=torch.float64, device=dev), mscale=mscale)
    seqs = q.KvSeqs(torch.tensor([0, 0, 1], **i32), pool.lens, pool.tables)
    parts = [model.qkv[i * H:(i + 1) * H].view(1, heads, dim) for i in range(3)]
    turned, att = (torch.empty(1, heads, dim, dtype=torch.float32, device=dev) for _ in range(2))
    work = torch.empty(q.qgemv_kv_attend_bytes(turned, seqs, cache), dtype=torch.uint8, device=dev)
    grown, one = torch.tensor([-1, n0], **i32), torch.tensor([0, 1], **i32)

    def token(only_attention=False):
        st = torch.cuda.current_stream().cuda_stream
        if not only_attention:
            grown.add_(one)
            q.qgemv_kv_resize(pool, cache, grown)
        for i, (mp, r, xp, yp, _, _, m, out_op) in enumerate(model.fcalls):
            if not only_attention:
                rc = model.lib.qgemv_rows_op(mp, 0, r, att.data_ptr() if m == 1 else xp, None, q.IN_RMS, model.eps,
                                             out_op, yp, 0, st)
                if rc != 0:
                    raise RuntimeError(f"qgemv_rows_op failed: {rc}")
            if m == 0:
                q.qgemv_kv_append(parts[1], parts[2], seqs, cache, i // 4, rope=rope, q=parts[0], q_out=turned)
                q.qgemv_kv_attend(turned, seqs, cache, i // 4, att, scale=dim ** -0.5, work=work)

    def replayed(f):
        if args.eager:
            return f
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        return graph.replay

    model.reset_fused()
    token()
    torch.cuda.synchronize()
    run = replayed(token)
    for _ in range(args.warmup):
        run()
    wall, _ = _timed(lambda i: run(), args.steps, torch)
    n = int(pool.lens[1])
    # the last layer's attention of the last token, in 64 bits
    k, v = (t[layers - 1][pool.tables[1, :-(-n // size)].long()].transpose(0, 1).reshape(heads, -1, dim)[:, :n].double()
            for t in (cache.k, cache.v))
    w = torch.softmax((k @ turned[0].double()[..., None])[..., 0] * dim ** -0.5, -1)
    want = (w[:, None] @ v)[:, 0]
    off = float((att[0].double() - want).abs().max() / want.abs().max())
    alone = replayed(lambda: token(only_attention=True))
    alone()
    wall_a, _ = _timed(lambda i: alone(), args.steps, torch)
    per = wall / args.steps
    return {"value": model.bytes_per_token / per / 1e9, "ms_per_step": per * 1e3, "tokens_per_s": 1 / per,
            "bytes_per_token": model.bytes_per_token, "cache_bytes_per_token": 2 * 2 * layers * n * H,
            "attention_ms_per_token": wall_a / args.steps * 1e3,
            "config": {"workload": c["name"] + "_context", "layers": layers, "format": FMT_LABEL[5], "heads": heads,
                       "head_dim": dim, "n_rot": rot, "context": n0, "cache": "f16, pages of 16",
                       "launch": "eager" if args.eager else "one HIP graph per token"},
            "parity": {"attention_max_rel": off, "tol": TOL, "length": n, "pass": bool(off <= TOL and n == total - 1)}}


def kquant_dense_workload(args, dev):
    """The dense 20B-class pass in the Q4_K_M mix: Q4_K QKV, out and up, Q6_K down."""
    return dense_workload(args, dev, cfg=6)


WORKLOADS = {"dense20b": dense_workload, "q4_0_4096": q4_0_workload, "moe_mxfp4": moe_workload,
             "ffn_streamed": ffn_streamed_workload, "q8_0_256": q8_0_small_workload,
             "q4_k_m_dense20b": kquant_dense_workload, "dense20b_batch": dense_batch_workload,
             "moe_streamed": moe_streamed_workload, "dense20b_context": dense_context_workload}


def extra_configs(args, dev):
    """The other workloads, each reduced to the figures it is quoted with, for
    the default run's line: Q8_0 256x1024 (latency, oracle parity), Q4_0
    4096x4096 (16-matrix grid, block_rows 0 vs 512), the streamed Q8_0 FFN trio
    (block_rows 128/512/2048 against the same run's pinned copy) and the MXFP4
    MoE (64 tokens, block_rows 0/128/512)."""
    import copy
    import torch
    out = {}
    a = copy.copy(args)
    a.warmup, a.steps = 2, 64
    t = time.perf_counter()
    r = q8_0_small_workload(a, dev)
    out["q8_0_256x1024"] = {"us_per_launch": r["ms_per_step"] * 1e3, "GBs_cache_resident": r["value"],
                            "parity": r.get("parity"), "note": r["config"]["note"]}
    r = q4_0_workload(a, dev)
    out["q4_0_4096x4096"] = {"GBs": r["value"], "pct_hbm_peak": r["pct_hbm_peak"],
                             "us_per_grid": r["ms_per_step"] * 1e3, "launch": r["config"]["launch"],
                             "sustained": r["sustained"], "single_matrix": r["single_matrix"],
                             "block_rows_0_vs_512_bit_identical": r["block_rows_0_vs_512_bit_identical"],
                             "sha256_y": r["sha256_y"], "parity": r.get("parity")}
    torch.cuda.empty_cache()
    a.steps = 8
    r = ffn_streamed_workload(a, dev)
    out["ffn_q8_0_streamed"] = {"link_GBs": r["value"], "pct_of_256MiB_copy": r["pct_of_256MiB_copy"],
                                "best_block_rows": r["config"]["best_block_rows"], "best_mode": r["best_mode"],
                                "h2d_256MiB_GBs": r["h2d_256MiB_GBs"], "lookahead": r["config"]["lookahead"],
                                "block_rows": r["block_rows"], "mapped": r["mapped"], "resident": r["resident"],
                                "sha256_y_resident": r["sha256_y_resident"]}
    torch.cuda.empty_cache()
    a.steps, a.block_rows = 0, 0
    r = moe_workload(a, dev)
    out["moe_mxfp4_top4"] = {"GBs": r["value"], "pct_hbm_peak": r["pct_hbm_peak"], "tokens_per_s": r["tokens_per_s"],
                             "us_per_token": r["us_per_token"], "bytes_per_token": r["bytes_per_token"],
                             "tokens": r["config"]["tokens"], "launches": r["config"]["launches_per_token"],
                             "block_rows_bit_identical": r["block_rows_bit_identical"],
                             "sha256_y_all_tokens": r["sha256_y_all_tokens"]}
    torch.cuda.empty_cache()
    out["extras_seconds"] = round(time.perf_counter() - t, 1)
    return out


# --- entry --------------------------------------------------------------------------

def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--gpus", type=int, default=1)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--warmup", type=int, default=2)
    p.add_argument("--workload", default="dense20b",
                   choices=sorted(WORKLOADS))
    p.add_argument("--layers", type=int, default=0, help="fewer layers for a quick run (not a valid headline)")
    p.add_argument("--chain", action="store_true",
                   help="dense pass as one chain launch per token (qgemv_chain_run) instead of 176 fused GEMV launches")
    p.add_argument("--eager", action="store_true",
                   help="issue each token's 176 fused launches from the host instead of replaying them as one HIP graph")
    p.add_argument("--graph", action="store_true", help="the default: one token's 176 fused launches replayed as a HIP graph")
    p.add_argument("--no-cpu-baseline", action="store_true")
    p.add_argument("--no-check", action="store_true")
    p.add_argument("--no-sustained", action="store_true",
                   help="q4_0_4096: leave out the 384 back-to-back grids timed for the sustained rate")
    p.add_argument("--no-extras", action="store_true",
                   help="dense20b only: skip the other workloads' figures and the read ceiling")
    p.add_argument("--no-free-running", action="store_true",
                   help="dense20b only: skip the oracle's own (free-running) pass of the first token")
    p.add_argument("--cpu-seconds", type=float, default=12.0)
    p.add_argument("--block-rows", type=int, default=0,
                   help="block_rows for moe_mxfp4; for ffn_streamed, the only block size to run (0 = 128/512/2048)")
    p.add_argument("--leg", default="all", choices=["all", "ring", "plan", "mapped"],
                   help="ffn_streamed: which streamed modes to run")
    p.add_argument("--batch", type=int, default=4, help="tokens per step of dense20b_batch")
    p.add_argument("--context", type=int, default=4096, help="cached positions of dense20b_context")
    p.add_argument("--kquant", action="store_true", help="dense20b_batch in the Q4_K_M mix")
    p.add_argument("--mfma", action="store_true",
                   help="dense20b_batch through qgemv_rows_mfma (fp32 matrix cores, 16 tokens per pass)")
    p.add_argument("--copy-calibration", action="store_true",
                   help="first run a 256 MiB device-to-device copy (a kernel of known traffic, to scale HBM counters)")
    args = p.parse_args(argv)
    if args.gpus != 1:
        print(f"bench.py: the benchmark runs on one GPU; --gpus {args.gpus} is not supported "
              "(splitting the rows over several GPUs is described in the design notes, not implemented)",
              file=sys.stderr)
        return 2
    import torch
    if not torch.cuda.is_available():
        print("bench.py: no GPU visible", file=sys.stderr)
        return 1
    dev = torch.device("cuda:0")
    if args.copy_calibration:
        src = torch.ones(256 << 20, dtype=torch.uint8, device=dev)
        dst = torch.empty_like(src)
        for _ in range(3):
            dst.copy_(src)
        torch.cuda.synchronize()
        del src, dst
    fn = WORKLOADS[args.workload]
    res = fn(args, dev)
    if args.workload in ("dense20b", "q4_k_m_dense20b") and not args.no_extras:
        ceil = read_ceiling(dev)
        res["read_ceiling"] = ceil
        res["pct_of_read_ceiling"] = 100.0 * res["value"] / ceil["GBs"]
        if args.workload == "dense20b":
            res.update(extra_configs(args, dev))
    line = {
        "metric": METRIC,
        "value": round(res.pop("value"), 3),
        "unit": "GB/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(res.pop("ms_per_step"), 4),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32",
        "data": "synthetic",
    }
    line.update(res)
    print(json.dumps(line), flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
