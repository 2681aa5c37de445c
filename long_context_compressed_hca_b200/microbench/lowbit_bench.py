"""Times the low-bit decode operators on the cases of perf/operators.py, from the repository's root.

    python -m long_context_compressed_hca_b200.microbench.lowbit_bench [NAME ...]          # device time per call, host time
    python -m long_context_compressed_hca_b200.microbench.lowbit_bench --once [NAME ...]   # one call each, for a profiler

Device time: 20 calls captured in a graph, the best of 10 replays by CUDA events (inputs below 126 MB stay in L2).  Host
time: from one call's start to the next's, nothing waited for.
"""
import sys
import time

import torch

import perf.operators as operators


def times(state, calls=20):
    for _ in range(3):
        operators.run(state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            operators.run(state)
    best = float("inf")
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / calls)
    t0 = time.perf_counter()
    for _ in range(200):
        operators.run(state)
    host = (time.perf_counter() - t0) / 200 * 1e6
    torch.cuda.synchronize()
    return best, host


def main(argv):
    operators.own = True
    names = [a for a in argv if not a.startswith("-")]
    for case in operators.listed():
        if names and case["name"] not in names:
            continue
        state = operators.prepare(case, 1)
        if "--once" in argv:
            operators.run(state)
            torch.cuda.synchronize()
            print(case["name"], "done", flush=True)
        else:
            device, host = times(state)
            work = operators.work(case)
            print(f"{case['name']:20s} device {device:8.2f} us  host {host:6.2f} us  {work['bytes'] / device / 1e3:7.0f} GB/s  "
                  f"{work['flops'] / device / 1e6:7.1f} TFLOP/s", flush=True)
        del state
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main(sys.argv[1:])
