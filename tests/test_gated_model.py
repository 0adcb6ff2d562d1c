"""The launch-time models behind the choices for integer and gated products and
for gradients: the constants compiled into the library are what the fit gives
on the committed times, the choices are near the fastest shape timed, and the
library picks what the Python model picks.  CPU only: config names come from
the library without a GPU."""
import json
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_bf16_amd", "csrc")


@pytest.fixture(scope="module")
def gm():
    import __graft_entry__

    b = __graft_entry__._load_builder()
    if not os.path.exists(b.LIB):
        b.build()
    from dense_gemm_bf16_amd import gated_model

    return gated_model


@pytest.fixture(scope="module")
def records(gm):
    with open(gm.DATA) as f:
        return json.load(f)


def compiled(gm):
    """{bytes: {shape: constants}} as written in gated_api.hip."""
    text = open(os.path.join(CSRC, "gated_api.hip")).read()
    number = r"([\d.]+)f?"
    five = r"\{%s, %s, %s, %s, %s\}" % ((number,) * 5)
    rows = re.findall(r"ROW\((\w+), [^{]*?(\d+),\s*%s, %s\)" % (five, five), text)
    out = {1: {}, 2: {}}
    for name, resident, *c in rows:
        assert gm.SHAPES[name][3] == int(resident), name
        out[1][name] = tuple(float(v) for v in c[:5])
        if name != gm.NOT_GATED:  # 16-bit products are gated ones
            out[2][name] = tuple(float(v) for v in c[5:])
    return out


def compiled_gradients():
    text = open(os.path.join(CSRC, "grad_api.hip")).read()
    out = {n: tuple(float(v) for v in c) for n, *c in
           re.findall(r'\{"(b\d+x\d+)", \d+, \d+, \d+, \d, ([\d.]+), ([\d.]+), ([\d.]+), &', text)}
    out["sum"] = tuple(float(v) for v in re.search(
        r"kSumUs = ([\d.]+), kSumUsPerMB = ([\d.]+), kTail = ([\d.]+);", text).groups())
    return out


def test_compiled_constants_are_the_fit(gm, records):
    assert len(records["products"]) == 591
    fitted, written = gm.fit(records["products"]), compiled(gm)
    for size in (1, 2):
        assert list(written[size]) == list(fitted[size])
        for shape, c in written[size].items():
            for digits, a, b in zip((3, 2, 2, 2, 2), fitted[size][shape], c):
                assert abs(a - b) <= 0.75 * 10 ** -digits, (size, shape, fitted[size][shape], c)


def test_choices_are_near_the_fastest(gm, records):
    quality = gm.choice_quality(compiled(gm), records["products"])
    for kind in gm.KINDS:
        q = [v for v, k in quality if k == kind]
        assert len(q) == 197 and gm.geomean(q) < 1.015 and max(q) < 1.35
    q = gm.grad_quality(compiled_gradients(), records["gradients"])
    assert len(q) == 100 and gm.geomean(q) < 1.0115 and max(q) < 1.25


def test_what_the_library_runs_is_timed_and_near_the_fastest(gm, records):
    """Two launches and shapes that the sweep left out among them."""
    import numpy as np

    c = {b: {s: tuple(float(np.float32(v)) for v in k) for s, k in by.items()}
         for b, by in compiled(gm).items()}
    assert sum("+" in p for r in records["choices"] for p in r["times"]) >= 11
    quality = gm.library_quality(c, records["products"], records["choices"])
    assert len(quality) == 591
    q = [v for v, _ in quality]
    print(gm.geomean(q), max(q))
    assert gm.geomean(q) < 1.013 and max(q) < 1.35


def test_shapes_are_those_built(gm):
    import dense_gemm_bf16_amd as g

    assert g.i8_config_names() == list(gm.SHAPES)


def test_library_picks_the_models_shape(gm):
    import numpy as np

    import dense_gemm_bf16_amd as g

    # (the library holds the constants in fp32)
    c = {b: {s: tuple(float(np.float32(v)) for v in k) for s, k in by.items()}
         for b, by in compiled(gm).items()}
    rng = np.random.default_rng(5)
    split = 0
    for i in range(1500):
        low = (1, 1, 1) if i < 1000 else (200, 2000, 64)
        M, N, K = (int(np.exp(rng.uniform(np.log(lo), np.log(hi))))
                   for lo, hi in zip(low, (9000, 30000, 17000)))
        kind = list(gm.KINDS)[i % 3]
        size, gated = gm.KINDS[kind]
        want = gm.choose(c[size], gated, M, N, K * size)
        got = g.i8_config_name(M, N, K) if kind == "i8" else \
            g.gated_config_name(g.GEMM_TYPE_I8 if size == 1 else g.GEMM_TYPE_F16, M, N, K)
        assert got == want, (kind, M, N, K)
        split += "+" in got
    assert split > 20


def test_library_picks_near_the_models_plan(gm, records):
    """The plan it names for the products that were timed is the model's
    cheapest of those it may take (at least four K-steps a slice), whose splits
    it makes even."""
    import dense_gemm_bf16_amd as g

    c = compiled_gradients()
    for r in records["gradients"]:
        M, F, K = r["M"], r["F"], r["K"]
        steps, best = (2 * -(-F // 64), -(-M // 64)), None
        for tile, (bm, _) in gm.TILES.items():
            tiles = (-(-M // bm) * -(-K // bm), 2 * -(-F // bm) * -(-K // bm))
            ways = [[s for s in (1, 2, 4, 8, 16) if s == 1 or (n // s >= 4 and t * s <= 1024)]
                    for n, t in zip(steps, tiles)]
            for sx in ways[0]:
                for sw in ways[1]:
                    us = gm.grad_us(c, M, F, K, f"{tile}_k{sx}_k{sw}")
                    if best is None or us < best[0]:
                        best = (us, tile, sx, sw)
        even = [-(-n // -(-n // s)) for n, s in zip(steps, best[2:])]
        assert g.gated_backward_config_name(M, F, K) == f"{best[1]}_k{even[0]}_k{even[1]}", (M, F, K)
