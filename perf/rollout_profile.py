"""Times behind the rollout operators' figures, of the kernels alone.

  rocprofv3 --kernel-trace --output-format csv -d DIR -o run -- python perf/rollout_profile.py run
      every case of perf/operators.py: three states each, 35 passes in rotation
  python perf/rollout_profile.py table DIR/run_kernel_trace.csv
      the trace as a table, kernel by kernel
  python perf/rollout_profile.py sizes [--only NAME,NAME]
      device time per call of the cases and of the sizes that the kernels' rules and comments
      name (a HIP graph of 12 calls over three states), and the two rates that floors are put at

A pass's dispatches are told apart from the preparation's by their names: between two cases some
kernel that is not this library's always runs.
"""
import argparse
import csv
import os
import statistics
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

PASSES, STATES, CALLS = 35, 3, 12


def sizes():
    """The listed cases, and the sizes that rules and comments name."""
    from perf import operators as o
    lin, att = o._linear, o._attention
    return o.listed() + [
        lin("65536x7168 by 1 row", "nv", 1, 65536, 7168),
        lin("65536x7168 by 16 rows", "nv", 16, 65536, 7168),
        lin("65536x7168 by 64 rows", "nv", 64, 65536, 7168),
        lin("8192x7168 by 64 rows", "nv", 64, 8192, 7168),
        lin("MXFP4 65536x7168 by 16 rows", "mx", 16, 65536, 7168),
        lin("4096x4096 by 8 rows", "nv", 8, 4096, 4096),
        lin("2048x2048 by 8 rows", "nv", 8, 2048, 2048),
        lin("1024x7168 by 8 rows", "nv", 8, 1024, 7168),
        lin("16384x2048 by 8 rows", "nv", 8, 16384, 2048),
        lin("2048x2048 by 24 rows", "nv", 24, 2048, 2048),
        lin("7168x2048 by 24 rows", "nv", 24, 7168, 2048),
        lin("MXFP4 32 experts, 256 rows", "mx", 256, 2048, 7168, experts=32),
        lin("32 experts, 1024 rows", "nv", 1024, 2048, 7168, experts=32),
        att("512 items of 512 tokens", 64, 1, 64, 8, 128, 64, 512, 512),
        att("2048 items of 30-500", 256, 1, 32, 8, 128, 64, 30, 500),
        att("512 items of 2000-4000", 64, 1, 32, 8, 128, 64, 2000, 4000),
        att("256 items of 1000-4000", 32, 1, 32, 8, 128, 64, 1000, 4000),
        att("64 items of 2000-4000", 8, 1, 32, 8, 128, 64, 2000, 4000),
        att("128 items of 100-700", 16, 1, 32, 8, 128, 16, 100, 700),
        att("one context of 32768", 1, 1, 32, 8, 128, 64, 32768, 32768),
        att("64 sequences x 64 rows, 512-2000", 64, 16, 32, 8, 128, 64, 512, 2000),
        att("4 sequences x 64 rows, 512-2000", 4, 16, 32, 8, 128, 64, 512, 2000),
        att("4 prompts of 8192, heads of 64", 64, 1, 32, 8, 64, 64, 64, 1024, groups=4, prefix=8192),
        att("4 prompts of 8192, heads of 256", 64, 1, 32, 8, 256, 64, 64, 1024, groups=4, prefix=8192),
        att("4 prompts of 8192 x 256 rows", 128, 1, 32, 4, 128, 64, 64, 1024, groups=4, prefix=8192),
        att("4 prompts of 16384 x 512 rows", 256, 1, 64, 8, 128, 64, 64, 1024, groups=4, prefix=16384),
        att("512 queries of 4 sequences, 512-4096", 4, 512, 32, 8, 128, 64, 512, 4096),
    ]


def states_of(case):
    from perf import operators as o
    o.own = False
    states = [o.prepare(case, seed) for seed in range(STATES)]
    o.own = True
    return o, states


def run(only):
    import torch
    from perf import operators as o
    for case in o.listed():
        if only and case["name"] not in only:
            continue
        o, states = states_of(case)
        torch.cuda.synchronize()
        for i in range(PASSES):
            o.run(states[i % STATES])
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        del states
        torch.cuda.empty_cache()


def table(path, only):
    from perf import operators as o
    rows = sorted(csv.DictReader(open(path)), key=lambda r: int(r["Start_Timestamp"]))
    cases, inside = [], False
    for r in rows:
        # the plain cache fill and quantizers of the package do not run here: preparation is torch's
        mine = "fp4q::" in r["Kernel_Name"]
        if mine and not inside:
            cases.append({})
        inside = mine
        if mine:
            name = r["Kernel_Name"].replace("fp4q::(anonymous namespace)::", "").replace("void ", "")
            grid = ",".join(r["Grid_Size_" + d] for d in "XYZ")
            us = (int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3
            cases[-1].setdefault((name.split("(")[0], grid), []).append(us)
    names = [c["name"] for c in o.listed() if not only or c["name"] in only]
    if len(names) != len(cases):
        sys.exit("%d cases in the trace, %d expected" % (len(cases), len(names)))
    print("| case | kernel | grid (work-items) | dispatches | p50 | min |\n|---|---|---|---|---|---|")
    for name, kernels in zip(names, cases):
        for (kernel, grid), us in kernels.items():
            print("| %s | `%s` | %s | %d | %.2f | %.2f |" % (
                name, kernel, grid, len(us), statistics.median(us), min(us)))


def device_us(torch, call):
    """Device time of call(i), i the call's number: a graph of CALLS of them, five times over."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for i in range(STATES):
            call(i)
    torch.cuda.synchronize()
    graph, keep = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph, stream=stream):
        for i in range(CALLS):
            keep.append(call(i))
    times = []
    for _ in range(7):
        graph.replay()
        torch.cuda.synchronize()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(4):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / (4 * CALLS))
    return statistics.median(times)


def print_sizes(only):
    import torch
    if not only:
        a = torch.randn((8192, 8192), device="cuda").bfloat16()
        us = device_us(torch, lambda i: a @ a)
        print("library's 8192^3 BF16 product: %.0f us, %.2f PFLOP/s" % (us, 2 * 8192 ** 3 / us / 1e9))
        big = torch.empty(1 << 28, device="cuda")
        out = torch.empty_like(big)
        us = device_us(torch, lambda i: out.copy_(big))
        print("torch's copy of 1 GiB: %.0f us, %.2f TB/s" % (us, 2 * big.numel() * 4 / us / 1e6))
        del a, big, out
    print("| size | us | floor us |\n|---|---|---|")
    for case in sizes():
        if only and case["name"] not in only:
            continue
        o, states = states_of(case)
        us = device_us(torch, lambda i: o.run(states[i % STATES]))
        work = o.work(case)
        floor = max(work["bytes"] / 6.42e6, work["flops"] / 1.2e9)
        print("| %s | %.2f | %.1f |" % (case["name"], us, floor), flush=True)
        del states
        torch.cuda.empty_cache()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("command", choices=("run", "table", "sizes"))
    ap.add_argument("trace", nargs="?")
    ap.add_argument("--only", default="")
    args = ap.parse_args()
    only = [n for n in args.only.split(",") if n]
    if args.command == "table":
        table(args.trace, only)
    elif args.command == "run":
        run(only)
    else:
        print_sizes(only)


if __name__ == "__main__":
    main()
