"""The launch-time model behind the choice of kernel shape for the e4m3 and
the experts' products.

``choose_block`` (``csrc/block_api.hip``) runs the shape whose launch the model
finds cheapest, or, for a dense product, two shapes side by side where that is
3 % cheaper.  This module holds the same model in Python, the sweep that times
every shape on the GPU, and the fit of the model's constants to those times,
so the constants compiled into the library can be derived again and checked.

Model of one launch (microseconds).  ``units`` workgroups run on CUs that hold
``resident`` of them each, in passes of 256 * resident.  A pass costs steps *
step + tile (steps: 128-byte K-steps of a wave group; tile: first loads and
epilogue); a last pass with a fraction f of its workgroups costs part + (1 -
part) * f of that; a launch adds base.  Reading B at 5.2 TB/s (and 2.5 us) is
a floor, joined as fourth powers (the fit counts a dense A as well, and the
experts' rows as they fell, which the library cannot know).  Each shape has
its four constants twice: one set for 16-bit operands and for e4m3 with a
16-bit C, one for e4m3 with an fp32 C, whose codes are widened to bf16 first.

Usage::

    python -m dense_gemm_bf16_amd.block_model sweep --out timings.json   # GPU
    python -m dense_gemm_bf16_amd.block_model fit                        # CPU

``fit`` reads ``plan_model_data/block_shapes.json``: 167 products (dense: M
1-4096, N x K from 600 x 1000 to 28672 x 1024; experts: 8 to 128 of them, 1 to
8192 tokens, e4m3 and bf16), each timed in the shapes that were in question,
with inputs that change from call to call.  One shape of it, ``b64x128`` (64 x
128 tiles, one wave group), was timed but not built: without it the choice
among the others loses 0.4 % more over all products.
"""
from __future__ import annotations

import argparse
import json
import math
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
DATA = os.path.join(_HERE, "plan_model_data", "block_shapes.json")
CUS = 256
STEP_BYTES = 128
SCALE_BLOCK = 128
STREAM_MB_PER_US, STREAM_BASE_US = 5.2, 2.5
SPLIT_GAIN = 0.97

# name -> (BM, BN, wave groups along K, workgroups a CU holds), in the
# library's order, which decides ties
SHAPES = {
    "b256x256": (256, 256, 1, 1),
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
}
# Not chosen for e4m3 with an fp32 C.  256 x 256 spills there (its widened
# fragments do not fit the registers): 4.9 us a K-step, where four 128 x 128
# tiles take 3.6.  256 x 128 was the fastest of all for one of the 24 products
# timed (2048 x 4096 x 4096: 60.0 us, 128 x 128 65.6) and up to 15 % slower
# on others; its times do not follow the model (13 % rms), which would take it
# for 777 x 10240 x 4104 (114.6 us, 128 x 128 99.7).
NEVER_WIDE = ("b256x256", "b256x128")


class Product:
    """Sizes of a product: dense (experts None), or R rows over that many."""

    def __init__(self, R, N, K, bytes=1, wide=False, experts=None, counts=None):
        self.R, self.N, self.K, self.bytes, self.wide = R, N, K, bytes, wide
        self.experts = experts
        self.counts = counts  # the rows of each expert, where they are known

    @classmethod
    def of(cls, record):
        r = record
        if r["op"] == "dense":
            return cls(r["M"], r["N"], r["K"], 1, r["out"] == "f32")
        e4m3 = r["type"] == "e4m3"
        return cls(r["R"], r["N"], r["K"], 1 if e4m3 else 2, e4m3 and r["out"] == "f32", r["E"],
                   r["counts"])

    def row_tiles(self, bm, known=False):
        """As the library counts them (or, `known`, from the experts' rows)."""
        if self.experts is None:
            return -(-self.R // bm)
        if known:
            return sum(-(-n // bm) for n in self.counts)
        used = min(self.R, self.experts)
        return max(self.R / bm + 0.5 * used, used)

    def b_rows(self, known=False):
        if self.experts is None:
            return 1
        return sum(n > 0 for n in self.counts) if known else min(self.R, self.experts)


def launch_us(constants, shape, p: Product, n=None, known=False) -> float:
    """Estimated time of a shape on n of the product's columns."""
    step, tile, part, base = constants
    bm, bn, groups, resident = SHAPES[shape]
    n = p.N if n is None else n
    passes, rest = divmod(p.row_tiles(bm, known) * -(-n // bn) / (CUS * resident), 1)
    if rest > 0:
        passes += part + (1 - part) * rest
    k_steps = -(-p.K * p.bytes // STEP_BYTES)
    t = passes * (-(-k_steps // groups) * step + tile) + base
    rows = p.b_rows(known) * n + (p.R if known and p.experts is None else 0)  # of K read
    floor = rows * p.K * p.bytes * 1e-6 / STREAM_MB_PER_US + STREAM_BASE_US
    return (t ** 4 + floor ** 4) ** 0.25


def cheapest(constants, p: Product, n=None, among=None):
    """(time, shape) of the cheapest shape; constants: {shape: four numbers}."""
    return min(((launch_us(constants[s], s, p, n), i, s) for i, s in enumerate(SHAPES)
                if s in constants and (among is None or s in among)))[::2]


def choose(constants, p: Product) -> str:
    """What the library runs, as its config name; constants: those of p.wide."""
    best, shape = cheapest(constants, p)
    name = shape
    if p.experts is not None or p.R < 1:
        return name
    best *= SPLIT_GAIN
    for s, (bm, bn, _, resident) in SHAPES.items():
        if s not in constants:
            continue
        rows, cols, one = -(-p.R // bm), -(-p.N // bn), CUS * resident
        if rows > one:
            continue
        head = rows * cols // one * one // rows * bn // SCALE_BLOCK * SCALE_BLOCK
        if not 0 < head < p.N:
            continue
        t = launch_us(constants[s], s, p, head)
        if t >= best:
            continue
        rest, tail = cheapest(constants, p, p.N - head)
        if t + rest < best:
            best, name = t + rest, f"{s}+{tail}"
    return name


def fit(records):
    """{False: {shape: constants}, True: those for e4m3 with fp32 C}: least
    squares on log time, each shape by itself."""
    from scipy.optimize import least_squares

    out = {}
    for wide in (False, True):
        out[wide] = {}
        for shape in SHAPES:
            if wide and shape in NEVER_WIDE:
                continue
            rows = []
            for r in records:
                p = Product.of(r)
                # (the shape for single tokens: where it is in question)
                few = p.experts is None and p.R <= 16
                if p.wide == wide and shape in r["times"] and (few or shape != "r16x16"):
                    rows.append((p, math.log(r["times"][shape])))
            if len(rows) < 8:
                if shape not in out[False]:
                    raise ValueError(f"too few times of {shape} to fit four constants")
                out[wide][shape] = out[False][shape]  # r16x16: bound by its loads, wide or not
                continue

            def of(v):
                return abs(v[0]), abs(v[1]), min(abs(v[2]), 1.0), abs(v[3])

            def off(v):
                return [math.log(launch_us(of(v), shape, p, known=True)) - us for p, us in rows]

            best = min((least_squares(off, [step, tile, part, 2.0])
                        for step in (0.3, 1.0) for tile in (1.0, 4.0) for part in (0.4, 0.8)),
                       key=lambda z: z.cost)
            out[wide][shape] = of(best.x)
    return out


def choice_quality(constants, records):
    """Time of the shape the model picks over the fastest shape timed (built
    or not), for each record; one launch only."""
    out = []
    for r in records:
        p = Product.of(r)
        _, pick = cheapest(constants[p.wide], p, among=r["times"])
        out.append((r["times"][pick] / min(r["times"].values()), p.wide))
    return out


def geomean(xs):
    xs = list(xs)
    return math.exp(sum(math.log(x) for x in xs) / len(xs))


# ------------------------------------------------------------------ timing

def _median_us(run, sets):
    """Median of three: time of a call among many, inputs in turn."""
    import torch

    def once(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for i in range(n):
            run(i % sets)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) * 1e3 / n

    once(3)
    n = max(5, min(200, int(8e3 / max(once(10), 1.0))))
    return sorted(once(n) for _ in range(3))[1]


def _codes(shape):
    import torch

    t = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        v = torch.randn(part.numel(), device="cuda", dtype=torch.bfloat16)
        part.copy_((v * 110).clamp_(-448, 448))
    return t


def _c(R, N, out):
    import torch

    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    return torch.empty((R, -(-N // 8) * 8), device="cuda", dtype=dtype)


def time_dense(M, N, K, out="bf16"):
    """Every shape's time for one dense product, as a record."""
    import torch

    import dense_gemm_bf16_amd as g

    kb, nb = -(-K // SCALE_BLOCK), -(-N // SCALE_BLOCK)
    sets = max(1, min(8, 600_000_000 // (N * K) + 1))
    ld = -(-K // 16) * 16
    A = [_codes((M, ld)) for _ in range(sets)]
    B = [_codes((N, ld)) for _ in range(sets)]
    SA, SB = torch.rand((kb, M), device="cuda"), torch.rand((nb, kb), device="cuda")
    C = _c(M, N, out)
    stream = torch.cuda.current_stream().cuda_stream
    args = [(M, N, K, A[i].data_ptr(), ld, SA.data_ptr(), M, B[i].data_ptr(), ld, SB.data_ptr(), kb,
             C.data_ptr(), C.stride(0), g._TYPES[C.dtype], stream) for i in range(sets)]
    times = {s: _median_us(lambda i: g._check(g._lib.gemm_fp8_ex(s.encode(), *args[i])), sets)
             for s in SHAPES}
    return dict(op="dense", M=M, N=N, K=K, out=out, times=times)


def time_experts(T, E, k, N, K, type="e4m3", out="bf16", skew=1.0):
    """The same for T tokens of k of E experts, unevenly loaded."""
    import torch

    import dense_gemm_bf16_amd as g

    unit = 16 if type == "e4m3" else 8
    ld, kb, nb, R = -(-K // unit) * unit, -(-K // SCALE_BLOCK), -(-N // SCALE_BLOCK), T * k
    sets = max(1, min(3, 2_000_000_000 // (E * N * ld * (16 // unit)) + 1))

    def draw(shape):
        if type == "e4m3":
            return _codes(shape)
        return torch.randn(shape, device="cuda", dtype=torch.bfloat16)

    A, B = [draw((T, ld)) for _ in range(sets)], [draw((E, N, ld)) for _ in range(sets)]
    SA = torch.rand((kb, T), device="cuda") if type == "e4m3" else None
    SB = torch.rand((E, nb, kb), device="cuda") if type == "e4m3" else None
    x = torch.randn((T, E), device="cuda") + skew * torch.randn((1, E), device="cuda")
    offsets, rows, _ = g.moe_plan(g.moe_route(x, k)[0], E)
    C = _c(R, N, out)
    stream = torch.cuda.current_stream().cuda_stream
    args = [(g._TYPES[A[i].dtype], R, N, K, E, T, A[i].data_ptr(), ld, g._ptr(SA), T,
             offsets.data_ptr(), rows.data_ptr(), B[i].data_ptr(), ld, N * ld, g._ptr(SB), kb,
             nb * kb, C.data_ptr(), C.stride(0), g._TYPES[C.dtype], stream)
            for i in range(sets)]
    times = {s: _median_us(lambda i: g._check(g._lib.gemm_moe_ex(s.encode(), *args[i])), sets)
             for s in SHAPES}
    counts = (offsets[1:] - offsets[:-1]).tolist()
    return dict(op="experts", R=R, E=E, N=N, K=K, type=type, out=out, counts=counts, times=times)


SWEEP_DENSE = [(N, K, out, Ms) for out, Ms, NKs in (
    ("bf16", (1, 8, 16, 32, 48, 64, 100, 128, 200, 256, 384, 512, 777, 1024, 1500, 2048, 3000, 4096),
     ((1024, 8192), (4096, 4096), (8192, 8192), (10240, 4104), (2048, 2048), (600, 1000))),
    ("bf16", (1, 24, 80, 160, 300, 600, 1200), ((28672, 1024), (3500, 6000))),
    ("f32", (1, 16, 64, 128, 300, 777, 2048), ((4096, 4096), (10240, 4104), (1024, 2048))))
    for N, K in NKs]
SWEEP_EXPERTS = [  # T, E, k, N, K, type, out, skew
    *((*s, "e4m3", "bf16", 1.0) for s in (
        (1, 128, 8, 4096, 2048), (4, 64, 4, 2048, 4096), (16, 128, 8, 4096, 2048),
        (64, 128, 8, 4096, 2048), (200, 128, 8, 2048, 2048), (500, 128, 4, 2048, 2048),
        (1000, 64, 4, 2048, 2048), (2000, 64, 4, 2048, 2048), (4000, 64, 4, 2048, 2048),
        (4096, 8, 2, 4096, 4096), (8192, 32, 4, 4096, 4096), (300, 16, 2, 1024, 1024),
        (1000, 16, 8, 512, 512), (4000, 100, 3, 700, 300))),
    *((*s, "bf16", "bf16", 0.5) for s in (
        (2, 8, 2, 14336, 4096), (16, 8, 2, 14336, 4096), (100, 8, 2, 14336, 4096),
        (300, 8, 2, 14336, 4096), (1000, 8, 2, 14336, 4096), (3000, 8, 2, 4096, 4096),
        (500, 64, 4, 2048, 1024))),
    *((*s, "e4m3", "f32", 1.0) for s in (
        (16, 64, 4, 2048, 2048), (500, 64, 4, 2048, 2048), (2000, 64, 4, 2048, 2048)))]


def sweep(out_path: str, every: int = 1) -> None:
    """Time every `every`-th product of the lists above on the GPU."""
    jobs = [(time_dense, (M, N, K, out)) for N, K, out, Ms in SWEEP_DENSE for M in Ms]
    jobs += [(time_experts, args) for args in SWEEP_EXPERTS]
    records = []
    for f, args in jobs[::every]:
        r = f(*args)
        records.append(r)
        best = min(r["times"], key=r["times"].get)
        print(f.__name__, args, f"{best} {r['times'][best]:.1f} us", flush=True)
        with open(out_path, "w") as file:
            json.dump(records, file)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    sub = ap.add_subparsers(dest="cmd", required=True)
    sw = sub.add_parser("sweep", help="time every shape on the GPU")
    sw.add_argument("--out", required=True)
    sw.add_argument("--every", type=int, default=1, help="only every n-th product")
    ft = sub.add_parser("fit", help="fit the constants and report the choice quality")
    ft.add_argument("--data", default=DATA)
    args = ap.parse_args(argv)
    if args.cmd == "sweep":
        sys.path.insert(0, os.path.dirname(_HERE))
        sweep(args.out, args.every)
        return 0
    with open(args.data) as f:
        records = json.load(f)
    constants = fit(records)
    for wide, by in constants.items():
        print("e4m3 with fp32 C" if wide else "16-bit C, or 16-bit operands")
        for shape, c in by.items():
            print(f"  {shape:12s} step {c[0]:.3f} tile {c[1]:.2f} part {c[2]:.2f} base {c[3]:.2f}")
    quality = choice_quality(constants, records)
    for wide in constants:
        q = [v for v, w in quality if w == wide]
        print(f"{len(q)} products: model's pick / fastest timed {geomean(q):.4f} "
              f"(worst {max(q):.3f})")
    return 0


if __name__ == "__main__":
    sys.exit(main())
