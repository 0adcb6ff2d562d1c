"""The launch-time model behind the choice of shape for the e4m3 and experts'
products: the constants compiled into the library are what the fit gives on
the committed times, and the library picks what the Python model picks.  CPU
only: config names come from the library without a GPU."""
import json
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
API = os.path.join(ROOT, "dense_gemm_bf16_amd", "csrc", "block_api.hip")


@pytest.fixture(scope="module")
def bm():
    import __graft_entry__

    b = __graft_entry__._load_builder()
    if not os.path.exists(b.LIB):
        b.build()
    from dense_gemm_bf16_amd import block_model

    return block_model


@pytest.fixture(scope="module")
def records(bm):
    with open(bm.DATA) as f:
        return json.load(f)


def compiled(bm):
    """{wide: {shape: constants}} as written in block_api.hip."""
    out = {False: {}, True: {}}
    four = r"\{([\d.]+)f, ([\d.]+)f, ([\d.]+)f, ([\d.]+)f\}"
    rows = re.findall(r'\{"(\w+)", (\d), (\d), %s, (?:%s|\{kNever, 0, 0, 0\})\}' % (four, four),
                      open(API).read())
    for name, groups, resident, *c in rows:
        assert bm.SHAPES[name][2:] == (int(groups), int(resident)), name
        out[False][name] = tuple(float(v) for v in c[:4])
        if c[4]:
            out[True][name] = tuple(float(v) for v in c[4:])
    return out


def test_compiled_constants_are_the_fit(bm, records):
    assert len(records) == 167
    fitted, written = bm.fit(records), compiled(bm)
    assert list(written[False]) == list(bm.SHAPES)
    assert [s for s in bm.SHAPES if s not in written[True]] == list(bm.NEVER_WIDE)
    for wide in written:
        for shape, c in written[wide].items():
            for digits, a, b in zip((3, 2, 2, 2), fitted[wide][shape], c):
                assert abs(a - b) <= 0.75 * 10 ** -digits, (wide, shape, fitted[wide][shape], c)


def test_choices_are_near_the_fastest_shape(bm, records):
    quality = bm.choice_quality(compiled(bm), records)
    narrow, wide = ([v for v, w in quality if w == x] for x in (False, True))
    assert len(narrow) == 143 and len(wide) == 24
    assert bm.geomean(narrow) < 1.0095 and max(narrow) < 1.185
    assert bm.geomean(wide) < 1.0205 and max(wide) < 1.245


def test_shapes_are_those_built(bm):
    import dense_gemm_bf16_amd as g

    assert g.fp8_config_names() == list(bm.SHAPES)


def test_library_picks_the_models_shape(bm):
    import numpy as np

    import dense_gemm_bf16_amd as g

    # (the library holds the constants in fp32)
    c = {w: {s: tuple(float(np.float32(v)) for v in k) for s, k in by.items()}
         for w, by in compiled(bm).items()}
    types = {"bf16": g.GEMM_TYPE_BF16, "f16": g.GEMM_TYPE_F16, "f32": g.GEMM_TYPE_F32}
    rng = np.random.default_rng(5)
    split = 0
    for i in range(2000):
        # (the last ones large and dense, where two shapes share a product)
        low = (0, 0, 0) if i < 1500 else (200, 4000, 64)
        R, N, K = (int(np.exp(rng.uniform(np.log(max(lo, 1)), np.log(hi))))
                   for lo, hi in zip(low, (9000, 30000, 17000)))
        E = None if i % 2 or i >= 1500 else int(np.exp(rng.uniform(0, np.log(300))))
        kind = "e4m3" if E is None else ("e4m3", "bf16", "f16")[i % 3]
        out = ("bf16", "f16", "f32")[i // 2 % 3]
        p = bm.Product(R, N, K, 1 if kind == "e4m3" else 2, kind == "e4m3" and out == "f32", E)
        want = bm.choose(c[p.wide], p)
        if E is None:
            got = g.fp8_config_name(R, N, K, types[out])
        else:
            type = g.GEMM_TYPE_E4M3 if kind == "e4m3" else types[kind]
            got = g.moe_config_name(type, R, N, K, E, types[out])
        assert got == want, (kind, out, R, N, K, E)
        split += "+" in got
    assert split > 50
