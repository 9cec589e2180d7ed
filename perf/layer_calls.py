"""Times calls of the operators between a decoder layer's products, or makes them for a profiler:

    python3 perf/layer_calls.py NAME[,NAME...] [--calls N] [--sets N] [--eager]

NAME: a case of more_operators.py (or cache_step, cache_prompt of operators.py), one of EXTRA's below, or "all".  A case's tensors are prepared
--sets times (default 3) and its calls go over the sets in turn.  Printed is the time of a call: one after another, and replayed in a graph.
With --eager nothing is timed: --calls calls (default 4), for counters.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_quantized_matvec_amd import ft  # noqa: E402
from perf import more_operators, operators  # noqa: E402

_norm = dict(op="norm", rows=8192, width=4096, kind="rms", post=False, residual=True, gate="none", scale=1.0, act="none", dtype="f32", pad=0)
_lora = dict(op="lora", tokens=512, order="runs", runs=1, k=4096, n=4096, adapters=48, rank=64, ragged=False, dtype="bf16", weights="bf16")
EXTRA = [
    dict(name="rope_normed", op="rope", tokens=6000, runs=3, heads=20, dim=128, rot=128, pairs="half", norm=True, n_pos=16384, dtype="bf16"),
    dict(_norm, name="norm_blocks", act="Q8_K"),
    dict(_norm, name="norm_8200", rows=2048, width=8200, dtype="bf16"),
    dict(_norm, name="norm_16384", rows=1024, width=16384, dtype="bf16"),
    dict(_norm, name="norm_16390", rows=1024, width=16390, dtype="bf16"),
    dict(_norm, name="norm_32768", rows=512, width=32768, dtype="bf16"),
    dict(_lora, name="lora_rank_100", tokens=1776, order="mixed", k=2048, n=1536, adapters=6, rank=100, dtype="f32"),
    dict(_lora, name="lora_pool_1", adapters=1),
    dict(_lora, name="lora_pool_48"),
]
TABLE = ("rope_table", 131072, 64)   # positions, pairs


def calls(name, sets):
    """A function per set of tensors."""
    if name == TABLE[0]:
        freqs = torch.tensor(ft.rope_freqs(2 * TABLE[2])[0], dtype=torch.float64, device="cuda")
        outs = [torch.empty(TABLE[1], 2 * TABLE[2], device="cuda") for _ in range(sets)]
        return [lambda o=o: ft.rope_table(TABLE[1], freqs, out=o) for o in outs]
    case = next(c for c in more_operators.listed() + EXTRA + operators.listed() if c["name"] == name)
    of = operators if case["op"] == "cache" else more_operators
    states = [of.prepare(case, i) for i in range(sets)]
    return [lambda s=s: of.run(s) for s in states]


def main():
    names = [c["name"] for c in more_operators.listed() + EXTRA] + [TABLE[0], "cache_step", "cache_prompt"]
    ap = argparse.ArgumentParser()
    ap.add_argument("names")
    ap.add_argument("--calls", type=int, default=0)
    ap.add_argument("--sets", type=int, default=3)
    ap.add_argument("--eager", action="store_true")
    a = ap.parse_args()
    more_operators.own = operators.own = True
    for name in names if a.names == "all" else a.names.split(","):
        fs = calls(name, a.sets)
        if a.eager:
            for i in range(a.calls or 4):
                fs[i % len(fs)]()
            torch.cuda.synchronize()
            print(name, flush=True)
            continue
        n = a.calls or 300
        for i in range(6):
            fs[i % len(fs)]()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for i in range(n):
            fs[i % len(fs)]()
        torch.cuda.synchronize()
        after = (time.perf_counter() - t) / n * 1e6
        stream, graph, per = torch.cuda.Stream(), torch.cuda.CUDAGraph(), 12
        ft.scratch_reserve(64 << 20, stream=stream)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for i in range(per):
                fs[i % len(fs)]()
        graph.replay()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        times = []
        for _ in range(5):
            start.record()
            for _ in range(max(1, n // per)):
                graph.replay()
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end) / max(1, n // per) / per * 1e3)
        print(f"{name:14s} {after:8.1f} us a call, {sorted(times)[2]:8.1f} us replayed", flush=True)
        del fs, graph
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
