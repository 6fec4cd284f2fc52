"""The kernels of the row-indexed products on perf/operators.py's listed cases: the program to
put under rocprofv3, and the table of profiles/rows_kernels.md from what it writes.

    P="python3 -m dense_gemm_nt_amd.profile_rows run"
    rocprofv3 --kernel-trace --output-format csv -d OUT -o trace -- $P
    rocprofv3 --pmc FETCH_SIZE --output-format csv -d OUT -o fetch -- $P
    rocprofv3 --pmc WRITE_SIZE --output-format csv -d OUT -o write -- $P
    rocprofv3 --pmc SQ_VALU_MFMA_BUSY_CYCLES GRBM_GUI_ACTIVE SQ_LDS_BANK_CONFLICT SQ_INSTS_VALU \\
        --output-format csv -d OUT -o sq -- $P
    python3 -m dense_gemm_nt_amd.profile_rows table OUT > profiles/rows_kernels.md

Every case is called CALLS times on three input sets in turn, of which the first
three calls are left out of the table; a device copy of COPY_MB MiB at the end
calibrates the byte counters.
"""
from __future__ import annotations

import csv
import importlib.util
import os
import re
import sys
from collections import OrderedDict

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS, WARM, COPY_MB = 33, 3, 512
SIMDS, XCDS = 1024, 8


def cases_module(name="operators"):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "perf", name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def run(cases="operators"):
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    import torch
    m = cases_module(cases)
    m.own = True
    for case in m.listed():
        states = [m.prepare(case, seed) for seed in range(3)]
        torch.cuda.synchronize()
        for i in range(CALLS):
            m.run(states[i % 3])
        torch.cuda.synchronize()
        print("profile_rows %s: %d calls" % (case["name"], CALLS), flush=True)
        del states
        torch.cuda.empty_cache()
    src = torch.ones(COPY_MB << 20, dtype=torch.uint8, device="cuda")
    dst = torch.empty_like(src)
    dst.copy_(src)
    torch.cuda.synchronize()


def _ours(name):
    return "gnt::" in name


def _short(name):
    name = re.sub(r"gnt::\(anonymous namespace\)::|gnt::|^void ", "", name)
    return name.split("(")[0]


def dispatches(path):
    """The dispatches of a rocprofv3 CSV in order: [{"name", "row", "counters"}], a
    counter file's several rows of one dispatch as one."""
    out = OrderedDict()
    with open(path, newline="") as f:
        for r in csv.DictReader(f):
            d = out.setdefault(int(r["Dispatch_Id"]), {"name": r["Kernel_Name"], "row": r, "counters": {}})
            if "Counter_Name" in r:
                d["counters"][r["Counter_Name"]] = float(r["Counter_Value"])
    return [out[k] for k in sorted(out)]


def segments(ds):
    """The unbroken runs of this library's kernels: one a case (what makes a case's inputs
    runs other kernels)."""
    runs, last = [], False
    for d in ds:
        ours = _ours(d["name"])
        if ours and not last:
            runs.append([])
        if ours:
            runs[-1].append(d)
        last = ours
    return runs


def _copy_scale(ds, counter):
    copies = [d for d in ds if not _ours(d["name"]) and ("copy" in d["name"].lower() or "elementwise" in d["name"])
              and d["counters"].get(counter)]
    return (COPY_MB << 20) / (copies[-1]["counters"][counter] * 1024.0)


def _blocks(r):
    return "x".join(str(int(r["Grid_Size_" + a]) // int(r["Workgroup_Size_" + a])) for a in "XYZ")


def table(folder, cases="operators", product=None):
    """The lines of the table: per case and kernel its median time and mean counters.  Where one
    kernel serves several products of a call, product(case, i, n) names the one of the i-th of
    its n launches in a call (None: they are one)."""
    files = {n: dispatches(os.path.join(folder, "%s_%s.csv" % (n, kind))) for n, kind in (
        ("trace", "kernel_trace"), ("fetch", "counter_collection"), ("write", "counter_collection"),
        ("sq", "counter_collection"))}
    runs = {n: segments(ds) for n, ds in files.items()}
    cases = cases_module(cases).listed()
    for n, s in runs.items():
        if [len(x) for x in s] != [len(x) for x in runs["trace"]] or len(s) != len(cases):
            raise SystemExit("%s holds other dispatches than the trace or the cases" % n)
    scale = {n: _copy_scale(files[n], c) for n, c in (("fetch", "FETCH_SIZE"), ("write", "WRITE_SIZE"))}
    out = []
    for i, case in enumerate(cases):
        sizes = ", ".join("%s %s" % (k, v) for k, v in case.items() if k != "name")
        out.append("| **%s** (%s) | | | | | | | |" % (case["name"], sizes))
        launches = OrderedDict()
        for j, d in enumerate(runs["trace"][i]):
            launches.setdefault((_short(d["name"]), _blocks(d["row"])), []).append(j)
        groups = OrderedDict()
        for (name, blocks), at in launches.items():
            n = len(at) // CALLS
            for k, j in enumerate(at):
                which = product(case, k % n, n) if product else None
                groups.setdefault((name + (": " + which if which else ""), blocks), []).append(j)
        for (name, blocks), at in groups.items():
            at = at[len(at) // CALLS * WARM:]
            ns = sorted(int(runs["trace"][i][j]["row"]["End_Timestamp"]) -
                        int(runs["trace"][i][j]["row"]["Start_Timestamp"]) for j in at)

            def mean(n, c):
                return sum(runs[n][i][j]["counters"][c] for j in at) / len(at)
            us = ns[len(ns) // 2] / 1e3
            read = mean("fetch", "FETCH_SIZE") * 1024 * scale["fetch"] / 1e6
            wrote = mean("write", "WRITE_SIZE") * 1024 * scale["write"] / 1e6
            busy = mean("sq", "SQ_VALU_MFMA_BUSY_CYCLES") / SIMDS / (mean("sq", "GRBM_GUI_ACTIVE") / XCDS)
            out.append("| %s | %s | %.1f | %.1f | %.1f | %.2f | %.0f %% | %.0f |" % (
                name, blocks, us, read, wrote, (read + wrote) / us, 100 * busy,
                mean("sq", "SQ_LDS_BANK_CONFLICT") / 1e3))
    return out, scale


HEAD = """# Kernels of the %(what)s

Traces and counters of `%(library)s`'s kernels on `perf/%(cases)s.py`'s listed cases, made by the commands in `dense_gemm_nt_amd/%(program)s.py` (each case's calls run %(calls)d times on three rotating input sets, the first three left out; median of the trace, mean of the counters, one run each).

Fabric bytes are the L2's requests to memory (FETCH_SIZE x %(fetch).3f, WRITE_SIZE x %(write).3f, as a device copy of %(copy)d MiB calibrates them). MFMA busy = SQ_VALU_MFMA_BUSY_CYCLES / %(simds)d SIMDs over GRBM_GUI_ACTIVE / %(xcds)d XCDs.

| kernel | blocks | µs | read MB | written MB | TB/s | MFMA busy | LDS bank conflicts (thousands) |
|---|---|---|---|---|---|---|---|"""


def heading(what, library, cases, program, scale):
    return HEAD % dict(what=what, library=library, cases=cases, program=program, calls=CALLS, fetch=scale["fetch"],
                       write=scale["write"], copy=COPY_MB, simds=SIMDS, xcds=XCDS)


def main():
    if sys.argv[1:] == ["run"]:
        run()
    elif len(sys.argv) == 3 and sys.argv[1] == "table":
        lines, scale = table(sys.argv[2])
        print(heading("products whose weight is picked per row", "libgemm_rows.so", "operators", "profile_rows", scale))
        print("\n".join(lines))
    else:
        raise SystemExit(__doc__)


if __name__ == "__main__":
    main()
