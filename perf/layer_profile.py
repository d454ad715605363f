"""Times behind the layer operators' figures, of the kernels alone.

  rocprofv3 --kernel-trace --output-format csv -d DIR -o run -- python perf/layer_profile.py run
      every case of perf/more_operators.py: three states each, 35 passes in rotation
  python perf/layer_profile.py table DIR/run_kernel_trace.csv
      the trace as a table, kernel by kernel
  python perf/layer_profile.py sizes [--only NAME,NAME]
      device time per call of the cases and of other sizes that comments name (a HIP graph of 12
      calls over three states), and the two rates that floors are put at
"""
import argparse
import csv
import os
import re
import statistics
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from perf import more_operators as ops  # noqa: E402
from perf.rollout_profile import PASSES, STATES, device_us  # noqa: E402

# the first kernel of a case
FIRST = ("rotary_kernel", "route_kernel", "dispatch_few", "count_chunks", "prompt_kernel")


def sizes():
    def prompt(text, tokens, dim, cached=0):
        return ops._prompt(text, 1, tokens, tokens, 32, 8, dim, cached=cached)
    return ops.listed() + [
        prompt("one prompt of 128", 128, 128),
        prompt("one prompt of 2048", 2048, 128),
        prompt("16 tokens behind 8000", 16, 128, cached=8000),
        prompt("8192 tokens, heads of 64", 8192, 64),
        prompt("4096 tokens, heads of 192", 4096, 192),
        prompt("4096 tokens, heads of 256", 4096, 256),
        ops._rows("512x2048, rows of 8", 512, 128, 8, 2048),
        ops._rows("1024x2048, rows of 8", 1024, 128, 8, 2048),
        ops._rows("16384x7168, rows of 8", 16384, 128, 8, 7168),
        ops._route("64 of 256, no bias", 64, 256, 8, "softmax"),
        ops._route("8192 of 256, bias and groups", 8192, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4),
    ]


def states_of(case):
    ops.own = False
    states = [ops.prepare(case, seed) for seed in range(STATES)]
    ops.own = True
    return states


def run(only):
    import torch
    for case in ops.listed():
        if only and case["name"] not in only:
            continue
        states = states_of(case)
        torch.cuda.synchronize()
        for i in range(PASSES):
            ops.run(states[i % STATES])
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        del states
        torch.cuda.empty_cache()


def table(path, only):
    rows = sorted(csv.DictReader(open(path)), key=lambda r: int(r["Start_Timestamp"]))
    times = {}
    for r in rows:
        if "fp4q" not in r["Kernel_Name"]:
            continue
        # (names with BF16 among their arguments come mangled or half demangled)
        name = re.search(r"(rotary_kernel|route_kernel|dispatch_few|count_chunks|place_chunks|copy_rows|"
                         r"combine_kernel|prompt_kernel|prompt_join)", r["Kernel_Name"]).group(1)
        grid = ",".join(r["Grid_Size_" + d] for d in "XYZ")
        us = (int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3
        times.setdefault((name, grid), []).append(us)
    names = [c["name"] for c in ops.listed() if not only or c["name"] in only]
    if len(names) != sum(kernel in FIRST for kernel, _ in times):
        sys.exit("the trace has not %d cases" % len(names))
    print("| case | kernel | grid (work-items) | dispatches | p50 | min |\n|---|---|---|---|---|---|")
    at = -1
    for (kernel, grid), us in times.items():
        at += kernel in FIRST
        print("| %s | `%s` | %s | %d | %.2f | %.2f |" % (
            names[at], kernel, grid, len(us), statistics.median(us), min(us)))


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
        states = states_of(case)
        us = device_us(torch, lambda i: ops.run(states[i % STATES]))
        work = ops.work(case)
        floor = max(work["bytes"] / 6.42e6, work["flops"] / 1.47e9)
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
