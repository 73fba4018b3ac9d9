"""Times the attention-side calls on the cases of perf/operators.py, or on sizes given.

    python examples/attention_times.py                                  every listed case
    python examples/attention_times.py --case cross_one_token           one of them
    python examples/attention_times.py --cross 4864x8192x8x8x128        rows x keys x heads x key heads x head width
    python examples/attention_times.py --case shared_block --calls 4    calls alone, nothing timed (for a profiler)

Two times of a call (us): by itself with a flushed L2 (median of 20, CUDA events around the call), and back to back in
bursts of 60 on three inputs in turn (the best of five; the stream is held up while a burst is issued, so that the host's
time counts only where it is longer than the GPU's by more than that).
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "perf"))

import torch

import operators


def cases(args):
    listed = {c["name"]: c for c in operators.listed()}
    picked = [listed[n] for n in args.case] if args.case else []
    for sizes in args.cross:
        rows, keys, hq, hk, d = (int(x) for x in sizes.split("x"))
        picked.append(dict(name=f"cross {sizes}", op="cross", rows=rows, keys=keys, hq=hq, hk=hk, d=d, segments=1, split=0,
                           valid=1.0, lse=False))
    return picked or list(listed.values())


def elapsed(what):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    what()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--case", action="append", default=[])
    ap.add_argument("--cross", action="append", default=[])
    ap.add_argument("--calls", type=int, default=0)
    args = ap.parse_args()
    operators.own = True
    flush = None if args.calls else torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    for case in cases(args):
        states = [operators.prepare(case, seed) for seed in range(1 if args.calls else 3)]
        for _ in range(args.calls or 3):
            for s in states:
                operators.run(s)
        torch.cuda.synchronize()
        if args.calls:
            continue
        alone = []
        for _ in range(20):
            flush.zero_()
            alone.append(elapsed(lambda: operators.run(states[0])))

        def burst():
            for i in range(60):
                operators.run(states[i % 3])
        bursts = []
        for _ in range(5):
            torch.cuda._sleep(4_000_000)
            bursts.append(elapsed(burst) / 60)
        work, t = operators.work(case), min(bursts)
        print(f"{case['name']:28s} alone {sorted(alone)[10]:9.1f} us   back to back {t:9.1f} us   "
              f"{work['bytes'] / t / 1e3:7.0f} GB/s  {work['flops'] / t / 1e6:7.1f} TFLOP/s", flush=True)


if __name__ == "__main__":
    main()
