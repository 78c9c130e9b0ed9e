"""Times of every kernel of the MXFP4 product over many sizes, and what its choice among them costs.

    python perf/mxfp4_product_choice.py time profiles/mxfp4_product_times.jsonl    # on a GPU, half a minute
    python perf/mxfp4_product_choice.py check profiles/mxfp4_product_times.jsonl   # anywhere

A line of the file is [m, k, n, {kernel: us, "chosen": us}]: calls in a graph over 2 to 24 states of more
than 400 MB together where 24 are enough for that (the 256 MB cache holds the small ones), the median
of five.  `check` reads the kernels' constants from the source, so it says what other constants would
choose on the same times."""

from __future__ import annotations

import json
import math
import os
import random
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

N_CU = 256
PROJECTIONS = [(4096, 4096), (6144, 4096), (14336, 4096), (28672, 4096), (4096, 14336), (2048, 7168), (1024, 4608),
               (4608, 1024), (512, 2048)]
TOKENS = [1, 4, 16, 32, 64, 128, 256, 512, 1024, 2048]


def sizes():
    """Projections at decode and prefill lengths, then sizes spread over their logarithms."""
    out = [(m, k, n) for m, k in PROJECTIONS for n in TOKENS]
    rng = random.Random(6)

    def spread(lo, hi):
        return round(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    while len(out) < len(PROJECTIONS) * len(TOKENS) + 430:
        m, k, n = spread(16, 14336), 32 * spread(2, 448), spread(1, 4096)
        if rng.random() < 0.7:
            k = max(64, k // 64 * 64)
        if rng.random() < 0.5:
            m = max(16, m // 16 * 16)
        if 2 * m * k * n < 3e11:
            out.append((m, k, n))
    return out


def kernels():
    """(rows, tokens, k groups, work groups per CU, k of a pass, whether k must be whole 64s, the four
    constants) of each kernel."""
    with open(os.path.join(ROOT, "gemv_prefill_decode_amd", "csrc", "gemm_mx.hip")) as f:
        src = f.read()
    number = r"([\d.]+)f?"
    rows = re.findall(r"\{(?:tiles|stream)<[^>]*>, (\d+), (\d+), (\d+), (\d+), (\d+), (true|false), "
                      + ", ".join([number] * 4) + r"\}", src)
    return [(*map(int, r[:5]), r[5] == "true", *map(float, r[6:])) for r in rows]


def predicted(kernel, m, k, n):
    rows, tokens, groups, per_cu, whole, _, start, step, step_per, end_per = kernel
    work = math.ceil(m / rows) * math.ceil(n / tokens)
    passes = math.ceil(math.ceil(k / whole) / groups)
    load = math.ceil(work / N_CU) if per_cu == 1 else max(1.0, work / N_CU)
    return start + passes * (step * math.ceil(work / (N_CU * per_cu)) + step_per * load) + end_per * load


def time(path):
    import torch

    import gemv_prefill_decode_amd as qmm
    table, stream = kernels(), torch.cuda.Stream()
    with open(path, "w") as f:
        for i, (m, k, n) in enumerate(sizes()):
            states = max(2, min(24, int(400e6 // (0.53 * (m + n) * k + 4 * m * n + 1))))

            def random_bytes(rows, width, lo, hi):
                return torch.randint(lo, hi, (rows, width), dtype=torch.uint8, device="cuda")

            held = [(random_bytes(m, k // 2, 0, 256), random_bytes(m, k // 32, 123, 128), random_bytes(n, k // 2, 0, 256),
                     random_bytes(n, k // 32, 123, 128), torch.empty(n, m, device="cuda")) for _ in range(states)]
            times = {}
            for j in list(range(len(table))) + ["chosen"]:
                if j != "chosen" and (table[j][5] and k % 64 or table[j][0] == 16 and 2 * m * k * n > 2e10):
                    continue        # cannot run, or is far behind
                os.environ.pop("QMM_MX_KERNEL", None)
                if j != "chosen":
                    os.environ["QMM_MX_KERNEL"] = str(j)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    for wq, we, xq, xe, out in held:
                        qmm.gemm_mxfp4(wq, we, xq, xe, out=out)
                begin, end, runs = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True), []
                for _ in range(6):
                    begin.record()
                    graph.replay()
                    graph.replay()
                    end.record()
                    end.synchronize()
                    runs.append(begin.elapsed_time(end) * 1e3 / 2 / states)
                times[str(j)] = round(sorted(runs[1:])[2], 2)
            f.write(json.dumps([m, k, n, times]) + "\n")
            f.flush()
            if i % 25 == 0:
                print(m, k, n, times, flush=True)


def check(path):
    table = kernels()
    with open(path) as f:
        lines = [json.loads(line) for line in f]
    loss, errors, chosen = [], [[] for _ in table], [0] * len(table)
    for m, k, n, times in lines:
        best = min(t for j, t in times.items() if j != "chosen")
        pick = min((predicted(x, m, k, n), j) for j, x in enumerate(table) if not (x[5] and k % 64))[1]
        chosen[pick] += 1
        loss.append((times.get(str(pick), times["chosen"]) / best, (m, k, n), pick))
        for j, t in times.items():
            if j != "chosen" and t < 1.7 * best:
                errors[int(j)].append(math.log(predicted(table[int(j)], m, k, n) / t))
    split = len(PROJECTIONS) * len(TOKENS)
    for name, part in (("projections", loss[:split]), ("spread sizes", loss[split:])):
        mean = math.exp(sum(math.log(x[0]) for x in part) / len(part))
        print(f"{name}: {len(part)}, the choice takes {100 * (mean - 1):.1f}% longer than the fastest, at most "
              f"{100 * (max(part)[0] - 1):.0f}% (m, k, n = {max(part)[1]})")
    for j, e in enumerate(errors):
        rms = math.sqrt(sum(x * x for x in e) / len(e)) if e else 0.0
        print(f"kernel {j} ({table[j][0]} x {table[j][1]}, {table[j][2]} k groups): chosen {chosen[j]} times, rms error "
              f"{100 * rms:.0f}% over {len(e)} sizes")


if __name__ == "__main__":
    {"time": time, "check": check}[sys.argv[1]](sys.argv[2])
