"""Profile of the paged cache's operators: every listed case of
perf/more_operators.py through the library, and a table of what rocprofv3 saw.

    cd /tmp && export TMPDIR=/tmp
    rocprofv3 --kernel-trace --stats --output-format csv -d t -o r -- python3 -u REPO/profiles/paged_cache_operators.py run 12
    rocprofv3 --pmc SET --output-format csv -d c0 -o r -- python3 -u REPO/profiles/paged_cache_operators.py run 3
    python3 REPO/profiles/paged_cache_operators.py table 12 3 t/r_kernel_trace.csv c*/r_counter_collection.csv

with the sets SETS below, each in a run of its own.  Times and bytes are those of a
pass, summed over a kernel's launches in it (some of which find nothing to do).
"""
import csv
import hashlib
import importlib.util
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SETS = ["SQ_BUSY_CYCLES SQ_VALU_MFMA_BUSY_CYCLES SQ_ACTIVE_INST_VALU SQ_LDS_IDX_ACTIVE GRBM_GUI_ACTIVE", "FETCH_SIZE",
        "WRITE_SIZE", "TCP_TCC_READ_REQ_sum"]
OURS = re.compile(r"^(void )?(qgemv_kv|\(anonymous namespace\))::(rope|append|attend|cut|resize|fork|move[sd]|copy)\w*kernel")


def cases():
    sys.path.insert(0, ROOT)
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "more_operators.py"))
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    return ops, ops.listed()


def run(passes):
    import torch
    ops, todo = cases()
    ops.own = True
    for case in todo:
        state = ops.prepare(case, 1)  # (torch's kernels here part the cases in the tables)
        torch.cuda.synchronize()
        for _ in range(passes):
            ops.run(state)
        torch.cuda.synchronize()
        print(case["name"], flush=True)


def launches(path):
    """Per case the library's launches: (kernel, its rows of the csv by launch)."""
    rows = sorted(csv.DictReader(open(path)), key=lambda r: int(r["Dispatch_Id"]))
    out, inside = [], False
    for r in rows:
        ours = OURS.search(r["Kernel_Name"])
        if ours and not inside:
            out.append([])
        inside = bool(ours)
        if ours:
            name = re.sub(r"\(anonymous namespace\)::|qgemv_kv::|void ", "", r["Kernel_Name"]).split("(")[0]
            out[-1].append((name, r))
    return out


def median(values):
    return sorted(values)[len(values) // 2]


def table(passes, counted, trace, counters):
    names = [c["name"] for c in cases()[1]]
    times, got = launches(trace), {}
    assert len(times) == len(names), (len(times), len(names))
    for path in counters:
        runs = launches(path)
        assert len(runs) == len(names), path
        for name, run_ in zip(names, runs):
            for kernel, r in run_:
                got.setdefault((name, kernel), {}).setdefault(r["Counter_Name"], []).append(float(r["Counter_Value"]))
    print("| case | kernel | launches | us a pass | median us | longest us | memory side read MB | written MB | L2 to L1 GB | "
          "MFMA | LDS | VALU |")
    print("|---|---|---|---|---|---|---|---|---|---|---|---|")
    for name, run_ in zip(names, times):
        for kernel in dict.fromkeys(k for k, _ in run_):
            us = [(int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3 for k, r in run_ if k == kernel]
            c = {k: sum(v) / counted for k, v in got[name, kernel].items()}
            cycles = c["GRBM_GUI_ACTIVE"] / 8  # of one XCD
            share = [c["SQ_VALU_MFMA_BUSY_CYCLES"] / (4 * 256 * cycles), c["SQ_LDS_IDX_ACTIVE"] / (256 * cycles),
                     c["SQ_ACTIVE_INST_VALU"] / (256 * cycles)]
            print(f"| {name} | `{kernel}` | {len(us) // passes} | {sum(us) / passes:.1f} | {median(us):.1f} | {max(us):.1f} | "
                  f"{c['FETCH_SIZE'] * 2048 / 1e6:.1f} | {c['WRITE_SIZE'] * 1024 / 1e6:.1f} | "
                  f"{c['TCP_TCC_READ_REQ_sum'] * 128 / 1e9:.2f} | " + " | ".join(f"{100 * s:.0f}%" for s in share) + " |")
    from quantized_gemv_gguf_amd import build
    h = hashlib.sha256()
    for path in build.kv_source_paths():
        h.update(open(path, "rb").read())
    print(f"\nkv_source_sha256 = {h.hexdigest()}")


if __name__ == "__main__":
    if sys.argv[1] == "run":
        run(int(sys.argv[2]))
    else:
        table(int(sys.argv[2]), int(sys.argv[3]), sys.argv[4], sys.argv[5:])
