"""Runs cases of perf/operators.py through the framework's calls: by the clock,
or under a profiler whose files it then sums up.

    python3 perf/profile_operators.py clock            us a pass, passes captured into one graph
    python3 perf/profile_operators.py run              the passes alone, for a profiler
    python3 perf/profile_operators.py table DIR        the profiler's csv files under DIR, by case and kernel

Each takes the same selection, and `table` the one of its `run`: --only NAME,NAME
for listed cases (all by default), any number of --case KEY=VALUE,... for others
(those alone, without --only).  A --case starts from a bf16 chain of 32 query and
8 kv heads of 128 on pages of 16; even=1 gives every request the same lengths.
Three sets of inputs are taken in turn."""
import argparse
import csv
import glob
import os
import re
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import perf.operators as M

DEFAULT = dict(op="tree", n_req=1, hq=32, hkv=8, dim=128, page=16, type="bf16", io="bf16", mask="chain")
RAGGED = M._plan


def _plan(case):
    if not case.get("even"):
        return RAGGED(case)
    n = case["n_req"]
    return np.full(n, case["prefix"], dtype=np.int64), np.full(n, case.get("rows", case.get("nodes")), dtype=np.int64)


def selected(args):
    out = [c for c in M.listed() if args.only is None and not args.case or c["name"] in (args.only or "").split(",")]
    for text in args.case:
        given = {k: int(v) if v.isdigit() else v for k, v in (x.split("=") for x in text.split(","))}
        out.append({**DEFAULT, "name": text, **given})
    return out


def states(case):
    made = [M.prepare(case, seed) for seed in range(3)]
    for s in made:
        M.run(s)
    torch.cuda.synchronize()
    return made


def clock(args):
    for case in selected(args):
        made, work = states(case), M.work(case)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(args.passes):
                M.run(made[i % 3])
        took = []
        for _ in range(9):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            graph.replay()
            end.record()
            torch.cuda.synchronize()
            took.append(begin.elapsed_time(end) * 1e3 / args.passes)
        us = sorted(took)[len(took) // 2]
        print(f"| {case['name']} | {us:.1f} us | {work['bytes'] / us / 1e6:.2f} TB/s | {work['flops'] / us / 1e6:.0f} TFLOP/s |", flush=True)


def run(args):
    for case in selected(args):
        made = states(case)
        for i in range(args.passes):
            M.run(made[i % 3])
        torch.cuda.synchronize()
        print("[case]", case["name"], flush=True)


def _dispatches(folder, pattern):
    """{column name: value} of each of the library's dispatches, in order."""
    rows = [r for f in glob.glob(os.path.join(folder, "**", pattern), recursive=True) for r in csv.DictReader(open(f))]
    return [r for r in rows if "dflash" in r["Kernel_Name"]]


def _kernel(name):
    return re.sub(r".*::(\w+)<([^>]*)>.*", r"`\1<\2>`", name)


def _by_case(args, dispatches):
    """(case, kernel, its dispatches): a pass of the attention is two of them."""
    at = 0
    for case in selected(args):
        n = (args.passes + 3) * (2 if case["op"] == "tree" else 1)
        mine, at = dispatches[at:at + n], at + n
        for kernel in dict.fromkeys(_kernel(d[0]["Kernel_Name"]) for d in mine):
            yield case, kernel, [d for d in mine if _kernel(d[0]["Kernel_Name"]) == kernel][-args.passes:]
    assert at == len(dispatches), (at, len(dispatches))


def table(args):
    trace = sorted(_dispatches(args.folder, "*kernel_trace.csv"), key=lambda r: int(r["Start_Timestamp"]))
    for case, kernel, mine in _by_case(args, [[r] for r in trace]) if trace else ():
        r = mine[0][0]
        us = sorted((int(d[0]["End_Timestamp"]) - int(d[0]["Start_Timestamp"])) / 1e3 for d in mine)
        shape = " | ".join(r[x] for x in ("Grid_Size_X", "Workgroup_Size_X", "VGPR_Count", "Accum_VGPR_Count", "LDS_Block_Size"))
        print(f"| {case['name']} | {kernel} | {shape} | {len(us)} | {us[0]:.1f} | {us[len(us) // 2]:.1f} | {us[-1]:.1f} |")
    groups = {}
    for r in _dispatches(args.folder, "*counter_collection.csv"):
        groups.setdefault(int(r["Dispatch_Id"]), []).append(r)
    for case, kernel, mine in _by_case(args, [groups[i] for i in sorted(groups)]) if groups else ():
        mean = {}
        for d in mine:
            for r in d:
                mean[r["Counter_Name"]] = mean.get(r["Counter_Name"], 0.0) + float(r["Counter_Value"]) / len(mine)
        print(f"| {case['name']} | {kernel} | " + " | ".join(f"{k} {v:.4g}" for k, v in sorted(mean.items())) + " |")


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("what", choices=["clock", "run", "table"])
    p.add_argument("folder", nargs="?")
    p.add_argument("--only")
    p.add_argument("--case", action="append", default=[])
    p.add_argument("--passes", type=int, default=30)
    args = p.parse_args()
    M.own, M._plan = True, _plan
    {"clock": clock, "run": run, "table": table}[args.what](args)


if __name__ == "__main__":
    main()
