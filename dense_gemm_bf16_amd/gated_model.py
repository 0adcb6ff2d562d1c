"""The launch-time models behind the choice of kernel shape for the integer and
gated products, and of tile and splits for the gradients.

``csrc/gated_api.hip`` runs the shape whose launch the first model finds
cheapest (or two shapes one after the other where that is 4 % cheaper),
``csrc/grad_api.hip`` the plan that the second finds cheapest.  This module
holds the same models in Python, the sweeps that time every shape and plan on
the GPU, and the fits of the models' constants to those times, so the constants
compiled into the library can be derived again and checked.

Products (microseconds).  ``units`` workgroups run on CUs that hold
``resident`` of them each, in passes of 256 * resident.  A pass costs steps *
step + tile (steps: 128-byte K-steps of a wave group; tile: first loads and
epilogue); a last pass with a fraction f of its workgroups, up to n of them on a
CU, costs part + stair * (n - 1) / (resident - 1) + (1 - part - stair) * f of
that; a launch adds base.  Reading B at 6.3 TB/s (and 2.2 us) is a floor, joined
as fourth powers.  Each shape has its five constants twice, for 8-bit integers
and for 16-bit types; a gated product counts B's rows, two for
each of its columns.  Least squares on log time, each shape by itself, over the
times within 2.5 of the product's fastest.

Gradients.  Both products share a launch; a workgroup's time is steps * step +
tile with ``resident`` of them on its CU.  A launch takes as long as its longest
workgroup, ``part`` to all of that by how full the GPU is, or as all of them
over the places there are, whichever is longer, and a split its sums' round
trip.  Its constants are not fitted to times alone but searched for the best
choice: the times of unlike plans lie closer than a model of them is off.

Usage::

    python -m dense_gemm_bf16_amd.gated_model sweep --out timings.json   # GPU
    python -m dense_gemm_bf16_amd.gated_model choices --out timings.json # GPU
    python -m dense_gemm_bf16_amd.gated_model fit                        # CPU
"""
from __future__ import annotations

import argparse
import json
import math
import os
import random
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
DATA = os.path.join(_HERE, "plan_model_data", "gated_shapes.json")
CUS = 256
STEP_BYTES = 128
STREAM_MB_PER_US, STREAM_BASE_US = 6.3, 2.2
SECOND_LAUNCH_US, SPLIT_GAIN = 2.5, 0.96

# name -> (rows of A, rows of B, wave groups along K, workgroups a CU holds),
# in the library's order, which decides ties
SHAPES = {
    "b256x256": (256, 256, 1, 1),
    "b256x192": (256, 192, 1, 1),
    "b256x128": (256, 128, 1, 1),
    "b128x128": (128, 128, 1, 2),
    "b128x128k2": (128, 128, 2, 1),
    "b64x128k2": (64, 128, 2, 1),
    "b64x64": (64, 64, 1, 2),
    "b64x64k2": (64, 64, 2, 1),
    "b32x128": (32, 128, 1, 2),
    "b32x64k4": (32, 64, 4, 1),
    "b32x32k4": (32, 32, 4, 1),
    "r16x16": (16, 16, 8, 4),
    "r16x8": (16, 8, 8, 4),
    "r32x16": (32, 16, 8, 4),
}
NOT_GATED = "b32x32k4"
# kind -> (bytes of an element, paired columns)
KINDS = {"i8": (1, False), "i8 gated": (1, True), "bf16 gated": (2, True)}


def launch_us(constants, shape, M, rows_b, k_bytes) -> float:
    step, tile, part, stair, base = constants
    bm, bn, groups, resident = SHAPES[shape]
    passes, rest = divmod(-(-M // bm) * -(-rows_b // bn), CUS * resident)
    if rest > 0:
        passes += part + stair * ((rest - 1) // CUS) / max(resident - 1, 1) + \
            (1 - part - stair) * rest / (CUS * resident)
    steps = -(-(-(-k_bytes // STEP_BYTES)) // groups)
    t = passes * (steps * step + tile) + base
    floor = rows_b * k_bytes * 1e-6 / STREAM_MB_PER_US + STREAM_BASE_US
    return (t ** 4 + floor ** 4) ** 0.25


def cheapest(constants, gated, M, rows_b, k_bytes):
    return min((launch_us(constants[s], s, M, rows_b, k_bytes), i, s) for i, s in enumerate(SHAPES)
               if s in constants and not (gated and s == NOT_GATED))[::2]


def choose(constants, gated, M, N, k_bytes) -> str:
    """What the library runs, as its config name; constants: those of the
    operands' type."""
    rows_b = 2 * N if gated else N
    best, name = cheapest(constants, gated, M, rows_b, k_bytes)
    if M < 1:
        return name
    best *= SPLIT_GAIN
    for s, (bm, bn, _, resident) in SHAPES.items():
        if s not in constants or (gated and s == NOT_GATED):
            continue
        rows, cols, one = -(-M // bm), -(-rows_b // bn), CUS * resident
        if rows > one:
            continue
        head = rows * cols // one * one // rows * bn // 128 * 128
        if not 0 < head < rows_b:
            continue
        t = launch_us(constants[s], s, M, head, k_bytes)
        if t >= best:
            continue
        rest, tail = cheapest(constants, gated, M, rows_b - head, k_bytes)
        if t + rest + SECOND_LAUNCH_US < best:
            best, name = t + rest + SECOND_LAUNCH_US, f"{s}+{tail}"
    return name


def fit(records):
    """{bytes: {shape: constants}} of the products' records."""
    from scipy.optimize import least_squares

    out = {}
    for size in (1, 2):
        out[size] = {}
        for shape in SHAPES:
            rows = []
            for r in records:
                b, gated = KINDS[r["kind"]]
                us, fastest = r["times"].get(shape), min(r["times"].values())
                if b == size and us is not None and us < 2.5 * fastest:
                    rows.append((r["M"], r["N"] * (2 if gated else 1), r["K"] * b, math.log(us),
                                 1.5 if us < 1.1 * fastest else 1.0))
            if len(rows) < 8:
                continue

            def of(v, many=SHAPES[shape][3] > 1):
                part = min(abs(v[2]), 1.0)
                return abs(v[0]), abs(v[1]), part, min(abs(v[4]), 1 - part) if many else 0.0, abs(v[3])

            def off(v):
                return [w * (math.log(launch_us(of(v), shape, M, n, kb)) - us)
                        for M, n, kb, us, w in rows]

            best = min((least_squares(off, (*x0, stair)) for x0 in (
                (0.5, 3, 0.6, 2), (1.5, 6, 0.7, 2), (0.3, 1, 0.3, 2.5), (2.4, 1.1, 0.3, 3))
                        for stair in (0.2,)), key=lambda z: z.cost)
            out[size][shape] = of(best.x)
    return out


def choice_quality(constants, records):
    """(time of the shape the model picks over the fastest, kind) of each
    product, among the shapes that the sweep timed: one launch only."""
    out = []
    for r in records:
        b, gated = KINDS[r["kind"]]
        among = {s: c for s, c in constants[b].items() if s in r["times"]}
        _, pick = cheapest(among, gated, r["M"], r["N"] * (2 if gated else 1), r["K"] * b)
        out.append((r["times"][pick] / min(r["times"].values()), r["kind"]))
    return out


def library_quality(constants, products, choices):
    """(time of what the library runs over the fastest of it and the shapes that
    were timed, kind) of each product.  What the sweep did not time (two launches,
    a shape that was not in question there) is in `choices`, timed beside the
    product's fastest shape."""
    later = {(r["kind"], r["M"], r["N"], r["K"]): r["times"] for r in choices}
    out = []
    for r in products:
        b, gated = KINDS[r["kind"]]
        name, times = choose(constants[b], gated, r["M"], r["N"], r["K"] * b), r["times"]
        if name not in times:
            times = later[r["kind"], r["M"], r["N"], r["K"]]
        out.append((times[name] / min(times.values()), r["kind"]))
    return out


def geomean(xs):
    xs = list(xs)
    return math.exp(sum(math.log(x) for x in xs) / len(xs))


# ------------------------------------------------------------------ gradients

# Where the search starts: the products' fits, and what a sum was seen to take.
START = {"b256x256": (1.34, 13.0, 0.8), "b128x128": (0.9, 7.0, 0.53), "sum": (3.5, 0.32, 0.15)}

# name -> (tile, workgroups a CU holds)
TILES = {"b256x256": (256, 1), "b128x128": (128, 2)}


def grad_us(constants, M, F, K, plan) -> float:
    """A gated product's gradients; constants: {tile: (step, tile, part)} and
    "sum": (us, us per MB, tail)."""
    tile, split_x, split_w = plan.split("_k")
    split_x, split_w = int(split_x), int(split_w)
    (bm, resident), (step, fixed, part) = TILES[tile], constants[tile]
    sum_us, per_mb, tail = constants["sum"]
    nx = -(-M // bm) * -(-K // bm) * split_x
    nw = 2 * -(-F // bm) * -(-K // bm) * split_w
    ux = -(-2 * -(-F // 64) // split_x) * step + fixed
    uw = -(-(-(-M // 64)) // split_w) * step + fixed
    places, longest = CUS * resident, max(ux, uw)
    fill = (nx + nw) / places
    us = longest * (part + (1 - part) * min(fill, 1))
    if fill > 1:
        us = max(us, (nx * ux + nw * uw) / places) + tail * longest
    if split_x > 1 or split_w > 1:
        ld = -(-K // 4) * 4
        mb = 4e-6 * ld * ((split_x * M if split_x > 1 else 0) + (split_w * 2 * F if split_w > 1 else 0))
        us += sum_us + per_mb * mb
    return us


def grad_quality(constants, records):
    """Time of the plan the model picks among those timed over the fastest."""
    out = []
    for r in records:
        pick = min(r["times"], key=lambda p: grad_us(constants, r["M"], r["F"], r["K"], p))
        out.append(r["times"][pick] / min(r["times"].values()))
    return out


def search(records, start, rounds=2500, seed=1):
    """Constants whose choice is best (losses count double where they are
    large) and whose times are not far off, which keeps them from values that
    choose well here and nowhere else; by random steps from `start`."""
    rng = random.Random(seed)
    names = list(TILES) + ["sum"]

    def loss(v):
        c = {n: v[3 * i:3 * i + 3] for i, n in enumerate(names)}
        q = [math.log(x) for x in grad_quality(c, records)]
        off = [math.log(grad_us(c, r["M"], r["F"], r["K"], p) / us) ** 2 for r in records
               for p, us in r["times"].items() if us < 1.3 * min(r["times"].values())]
        return sum(x * (1 + 2 * x) for x in q) / len(q) + 0.2 * sum(off) / len(off)

    v = [x for n in names for x in start[n]]
    best = loss(v)
    for _ in range(rounds):
        n = [x * math.exp(rng.gauss(0, 0.12)) if rng.random() < 0.4 else x for x in v]
        n[2], n[5] = min(n[2], 1.0), min(n[5], 1.0)
        new = loss(n)
        if new <= best:
            v, best = n, new
    return {n: tuple(v[3 * i:3 * i + 3]) for i, n in enumerate(names)}


# ------------------------------------------------------------------ timing

SWEEP = [(N, K) for N, K in ((8192, 8192), (28672, 4096), (4096, 4096), (2048, 1024), (600, 1000),
                             (10002, 2056), (1024, 8192), (1024, 4096), (512, 1024), (2000, 128),
                            (9000, 320))]
SWEEP_M = (1, 6, 16, 24, 32, 48, 64, 100, 128, 200, 256, 400, 512, 777, 1024, 1500, 2048, 4096)
SWEEP_GRADS = [(1000, 1365, 520), (100, 2000, 700), (8192, 1024, 1024), (2048, 2048, 1024),
               (512, 5001, 2055), (4096, 2048, 512), (16, 4096, 2048), (1, 1000, 1000),
               (333, 8000, 4096), (2048, 5461, 2048), (1024, 14336, 4096), (4096, 5376, 2048),
               (1, 14336, 4096), (16, 14336, 4096), (64, 14336, 4096), (200, 14336, 4096),
               (512, 14336, 4096), (4, 8192, 8192), (128, 8192, 8192), (32, 10000, 5000)]


def _replay_us(run, sets):
    """Best of three: time of a call among 2 * sets in a captured graph, inputs
    in turn."""
    import torch

    run(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(2 * sets):
            run(i % sets)
    graph.replay()
    best = math.inf
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / (2 * sets))
    return round(best, 2)


def _rows(shape, dtype, unit):
    import torch

    return torch.empty((shape[0], -(-shape[1] // unit) * unit), device="cuda", dtype=dtype)[:, :shape[1]]


def time_product(kind, M, rows_b, K, plans=None):
    """The times of one product in every shape that is in question, or as the
    plans named (two launches: only what the library chooses)."""
    import torch

    import dense_gemm_bf16_amd as g

    size, gated = KINDS[kind]
    sets = max(2, min(12, 600_000_000 // (rows_b * K * size) + 1))
    if size == 1:
        A = [_rows((M, K), torch.int8, 16).random_(-127, 128) for _ in range(sets)]
        B = [_rows((rows_b, K), torch.int8, 16).random_(-127, 128) for _ in range(sets)]
        SA, SB = torch.full((M,), 1e-3, device="cuda"), torch.full((rows_b,), 1e-3, device="cuda")
    else:
        A = [_rows((M, K), torch.bfloat16, 8).normal_() for _ in range(sets)]
        B = [_rows((rows_b, K), torch.bfloat16, 8).normal_() for _ in range(sets)]
    N = rows_b // 2 if gated else rows_b
    C = _rows((M, N), torch.bfloat16, 8)

    def run(i, shape):
        if kind == "i8":
            g.matmul_int8(A[i], SA, B[i], SB, config=shape, out=C)
        elif kind == "i8 gated":
            g.gated_matmul_int8(A[i], SA, B[i], SB, config=shape, out=C)
        else:
            g.gated_matmul(A[i], B[i], config=shape, out=C)

    times = {}
    for plan in plans or ():
        times[plan] = _replay_us(lambda i: run(i, None if "+" in plan else plan), sets)
    for shape, (bm, _, _, _) in SHAPES.items() if plans is None else ():
        if (gated and shape == NOT_GATED) or M > 64 * bm or (bm >= 256 and M <= 64) or \
                (shape[0] == "r" and M > 400):
            continue
        times[shape] = _replay_us(lambda i: run(i, shape), sets)
    return dict(kind=kind, M=M, N=N, K=K, times=times)


def time_grads(M, F, K):
    """The times of a gated product's gradients in every plan in question."""
    import torch

    import dense_gemm_bf16_amd as g

    x, W = _rows((M, K), torch.bfloat16, 8).normal_(), _rows((2 * F, K), torch.bfloat16, 8).normal_()
    dh = _rows((M, F), torch.bfloat16, 8).normal_()
    _, kept = g.gated_matmul(x, W, save=True)
    dx, dw = _rows((M, K), torch.bfloat16, 8), _rows((2 * F, K), torch.bfloat16, 8)
    times = {}
    for tile, (bm, _) in TILES.items():
        nx, nw = -(-M // bm) * -(-K // bm), 2 * -(-F // bm) * -(-K // bm)
        for sx in (1, 2, 4, 8, 16):
            for sw in (1, 2, 4, 8, 16):
                if (sx > 1 and (2 * -(-F // 64) // sx < 3 or nx * sx > 1024)) or \
                        (sw > 1 and (-(-M // 64) // sw < 3 or nw * sw > 1024)) or \
                        (M * F * K > 2 ** 38 and sx * sw > 1):
                    continue
                plan = f"{tile}_k{sx}_k{sw}"
                times[plan] = _replay_us(lambda i: g.gated_matmul_backward(
                    dh, x, W, kept, dx=dx, dw=dw, config=plan), 3)
    return dict(M=M, F=F, K=K, times=times)


def sweep(out_path: str, every: int = 1) -> None:
    rng = random.Random(3)

    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    grads = SWEEP_GRADS + [(log(1, 8192), log(256, 14336), log(128, 4096)) for _ in range(80)]
    data = dict(products=[], gradients=[])
    for kind in KINDS:
        for N, K in SWEEP[::every]:
            for M in SWEEP_M[::every]:
                if M * N * K > 2 ** 38:
                    continue
                r = time_product(kind, M, N, K)
                data["products"].append(r)
                best = min(r["times"], key=r["times"].get)
                print(kind, M, N, K, best, r["times"][best], "us", flush=True)
    for args in grads[::every]:
        r = time_grads(*args)
        data["gradients"].append(r)
        best = min(r["times"], key=r["times"].get)
        print("gradients", *args, best, r["times"][best], "us", flush=True)
    with open(out_path, "w") as f:
        json.dump(data, f, separators=(",", ":"))


def time_choices(path: str, out_path: str) -> None:
    """Adds `choices` to the sweep's data."""
    import dense_gemm_bf16_amd as g

    with open(path) as f:
        data = json.load(f)
    data["choices"] = []
    for r in data["products"]:
        kind, M, N, K, timed = r["kind"], r["M"], r["N"], r["K"], r["times"]
        size, gated = KINDS[kind]
        name = g.gated_config_name(g.GEMM_TYPE_I8 if size == 1 else g.GEMM_TYPE_BF16, M, N, K) if gated \
            else g.i8_config_name(M, N, K)
        if name not in timed:
            c = time_product(kind, M, 2 * N if gated else N, K, (name, min(timed, key=timed.get)))
            data["choices"].append(c)
            print(kind, M, N, K, c["times"], flush=True)
    with open(out_path, "w") as f:
        json.dump(data, f, separators=(",", ":"))


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    sub = ap.add_subparsers(dest="cmd", required=True)
    sw = sub.add_parser("sweep", help="time every shape and plan on the GPU")
    sw.add_argument("--out", required=True)
    sw.add_argument("--every", type=int, default=1, help="only every n-th size")
    ch = sub.add_parser("choices", help="time what the library chooses and the sweep did not time")
    ch.add_argument("--data", default=DATA)
    ch.add_argument("--out", required=True)
    ft = sub.add_parser("fit", help="fit the constants and report the choice quality")
    ft.add_argument("--data", default=DATA)
    args = ap.parse_args(argv)
    if args.cmd == "sweep":
        sys.path.insert(0, os.path.dirname(_HERE))
        sweep(args.out, args.every)
        return 0
    if args.cmd == "choices":
        time_choices(args.data, args.out)
        return 0
    with open(args.data) as f:
        data = json.load(f)
    constants = fit(data["products"])
    for size, by in constants.items():
        print("8-bit integers" if size == 1 else "16-bit types")
        for shape, c in by.items():
            print(f"  {shape:12s} step {c[0]:.3f} tile {c[1]:.2f} part {c[2]:.2f} "
                  f"stair {c[3]:.2f} base {c[4]:.2f}")
    quality = choice_quality(constants, data["products"])
    for kind in KINDS:
        q = [v for v, k in quality if k == kind]
        print(f"{kind}: {len(q)} products, model's pick / fastest timed {geomean(q):.4f} "
              f"(worst {max(q):.3f})")
    q = [v for v, _ in library_quality(constants, data["products"], data["choices"])]
    print(f"as the library runs them: {geomean(q):.4f} (worst {max(q):.3f})")
    half = data["gradients"][::2]
    found = search(half, START)
    print("gradients", {n: tuple(round(x, 3) for x in c) for n, c in found.items()})
    for name, rs in (("searched on", half), ("others", data["gradients"][1::2])):
        q = grad_quality(found, rs)
        print(f"  {name}: {len(q)}, model's pick / fastest timed {geomean(q):.4f} (worst {max(q):.3f})")
    return 0


if __name__ == "__main__":
    sys.exit(main())
