"""Times of the operators' listed cases (perf/operators.py), and summaries of rocprofv3's output on them.

    python perf/time_operators.py [--plain] [--only NAME,NAME]        us of a call among others, Python included
    python perf/time_operators.py --calls 30 [--only NAME,NAME]       that many calls of each case and nothing else: the program to profile
    python perf/time_operators.py --trace CSV                         summary of a kernel trace
    python perf/time_operators.py --counters CSV [--kernel NAME]      mean counters of a kernel's grids

Inputs go round three sets, so that a call does not find its own in the nearest cache. What the sets of a case hold together decides whether
they come from HBM: up to 256 MB they may stay in the memory-side cache, as a small model's weights do.
"""
import argparse
import collections
import csv
import importlib.util
import os
import statistics
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
SETS = 3


def cases(own, only):
    import torch

    spec = importlib.util.spec_from_file_location("operators", os.path.join(HERE, "operators.py"))
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    ops.own = own
    for case in ops.listed():
        if only and case["name"] not in only:
            continue
        states = [ops.prepare(case, seed) for seed in range(SETS)]
        torch.cuda.synchronize()
        yield case["name"], lambda i: ops.run(states[i % SETS])
        torch.cuda.synchronize()
        del states
        torch.cuda.empty_cache()


def time_calls(call, rounds=11, least_ms=20.0):
    """us a call, over rounds of calls that go on for about least_ms: median, least and longest."""
    import torch

    def run(n):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for i in range(n):
            call(i)
        end.record()
        end.synchronize()
        return start.elapsed_time(end) / n

    run(SETS)
    n = max(6, int(least_ms / run(6)))
    times = [run(n) * 1e3 for _ in range(rounds + 2)][2:]
    return statistics.median(times), min(times), max(times)


def short(name):
    return name.replace("fp4::(anonymous namespace)::", "").replace("void ", "").split("(")[0]


def trace(path):
    found = collections.defaultdict(list)
    with open(path) as f:
        for r in csv.DictReader(f):
            if "fp4::" in r["Kernel_Name"]:
                key = (short(r["Kernel_Name"]), int(r["Grid_Size_X"]) * int(r["Grid_Size_Y"]) * int(r["Grid_Size_Z"]),
                       int(r["Workgroup_Size_X"]), r["LDS_Block_Size"], r["VGPR_Count"], r["Scratch_Size"])
                found[key].append((int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3)
    print(f"{'kernel':60s} {'grid':>10s} {'group':>5s} {'LDS':>6s} {'VGPR':>5s} {'scratch':>7s} {'calls':>6s} {'median us':>9s} {'least us':>9s}")
    for k, v in found.items():
        print(f"{k[0]:60s} {k[1]:10d} {k[2]:5d} {k[3]:>6s} {k[4]:>5s} {k[5]:>7s} {len(v):6d} {statistics.median(v):9.2f} {min(v):9.2f}")


def counters(path, kernel):
    found = collections.defaultdict(list)
    with open(path) as f:
        for r in csv.DictReader(f):
            if "fp4::" in r["Kernel_Name"] and kernel in short(r["Kernel_Name"]):
                found[short(r["Kernel_Name"]), int(r["Grid_Size"]), r["Counter_Name"]].append(float(r["Counter_Value"]))
    for (name, grid, counter), v in found.items():
        print(f"{name:44s} {grid:10d} {counter:28s} {statistics.mean(v):16.0f}  over {len(v)} dispatches")


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--plain", action="store_true", help="the plain forms in place of the kernels")
    p.add_argument("--only", default="")
    p.add_argument("--calls", type=int, default=0)
    p.add_argument("--trace")
    p.add_argument("--counters")
    p.add_argument("--kernel", default="")
    a = p.parse_args()
    if a.trace:
        return trace(a.trace)
    if a.counters:
        return counters(a.counters, a.kernel)
    if not a.calls:
        print(f"{'case':20s} {'median us':>10s} {'least':>10s} {'longest':>10s}")
    for name, call in cases(not a.plain, set(filter(None, a.only.split(",")))):
        if a.calls:
            for i in range(a.calls):
                call(i)
            print(name, flush=True)
        else:
            print("{:20s} {:10.2f} {:10.2f} {:10.2f}".format(name, *time_calls(call)), flush=True)


if __name__ == "__main__":
    main()
