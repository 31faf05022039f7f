#!/usr/bin/env python3
"""Runs one hot-path entry point a few times on a named seeded workload, for profiler
captures (ncu) of a single kernel on a known case.  Exits 0 when every call returned
PKM_OK and the device status word stayed 0.  With --case the call is that of a case of
perf/more_operators.py (the paged K/V cache), whose calls raise an error otherwise.

  python tests/profile_case.py --workload deepseek_v3_bf16_decompress --launches 4
  python tests/profile_case.py --case token_batch --launches 2
"""
from __future__ import annotations

import argparse
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)


def main():
    import torch
    import workloads
    from gpu_util import DeviceCacheWrite, DeviceDecompress, DeviceKvMatmul

    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="deepseek_v3_bf16_decompress",
                    choices=sorted(workloads.WORKLOADS))
    ap.add_argument("--case", help="of perf/more_operators.py, instead of a workload")
    ap.add_argument("--launches", type=int, default=4)
    args = ap.parse_args()
    if args.case:
        from perf import more_operators
        more_operators.own = True
        case = {c["name"]: c for c in more_operators.listed()}[args.case]
        state = more_operators.prepare(case, 1)
        for _ in range(args.launches):
            more_operators.run(state)
        torch.cuda.synchronize()
        print(f"{args.case}: {args.launches} calls")
        return
    w = workloads.WORKLOADS[args.workload]()
    if args.workload.startswith("kv_matmul"):
        g = DeviceKvMatmul(w)
    elif args.workload.startswith("cache_write"):
        g = DeviceCacheWrite(w)
    else:
        g = DeviceDecompress(w, fp8=w.w_k_e4m3 is not None)
    for _ in range(args.launches):
        g.run()
    torch.cuda.synchronize()
    status = int(g.status.item())
    print(f"{args.workload}: {args.launches} calls, device status {status}")
    sys.exit(0 if status == 0 else 1)


if __name__ == "__main__":
    main()
