"""Calls the listed cases of operators.py through the library, for a profiler or a clock.

    python3 perf/drive.py [--only NAME,NAME] [--calls N]          N calls of each case (for rocprofv3)
    python3 perf/drive.py --time [--only ...] [--calls N]          median kernel time of N calls, by the
                                                                  library's own timing events
    python3 perf/drive.py --more [--only ...] [--calls N]          N passes of the cases of
                                                                  more_operators.py (for rocprofv3)

Two or three sets of inputs take turns, so that no call finds the last one's in the caches.  What counts is
the kernel alone: E4M3 outputs are not turned into values here.
"""
import argparse
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import more_operators  # noqa: E402
import operators  # noqa: E402
from combine_topk_idx_multihot_amd import binding as B  # noqa: E402


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--only", default="", help="names of cases, separated by commas")
    ap.add_argument("--calls", type=int, default=12)
    ap.add_argument("--time", action="store_true")
    ap.add_argument("--more", action="store_true")
    args = ap.parse_args()
    names = args.only.split(",") if args.only else None
    operators.own = more_operators.own = True
    if args.more:
        for case in more_operators.listed():
            if names and case["name"] not in names:
                continue
            sets = [more_operators.prepare(case, 1 + i) for i in range(3)]
            for i in range(args.calls):
                more_operators.run(sets[i % len(sets)])
            torch.cuda.synchronize()
            print(f"{case['name']}: {args.calls} passes", flush=True)
            del sets
            torch.cuda.empty_cache()
        return
    for case in operators.listed():
        if names and case["name"] not in names:
            continue
        sets = [operators.prepare(case, 1 + i) for i in range(3 if args.time else 2)]
        timer, us = B.KernelTimer() if args.time else None, []
        torch.cuda.synchronize()
        for i in range(args.calls):
            s = sets[i % len(sets)]
            if timer:
                timer.arm()
            s["call"](s["R"])
            if timer:
                torch.cuda.synchronize()
                us.append(timer.elapsed_ms() * 1e3)
        torch.cuda.synchronize()
        if timer:
            us = sorted(us[len(sets):] or us)
            m, w = us[len(us) // 2], operators.work(case)
            print(f"{case['name']:28s} {m:9.2f} us  {w['bytes'] / m / 1e6:6.2f} TB/s  "
                  f"{w['flops'] / m / 1e6:7.1f} TFLOP/s", flush=True)
        else:
            print(f"{case['name']}: {args.calls} calls", flush=True)
        del sets, s
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
