"""Routing, plan, experts' products and combine on the GPU against 64-bit
forms, and the layer they make."""
import numpy as np
import pytest

import block_ref as ref
from block_ref import block_product, check_rounded, dtype, padded

pytestmark = pytest.mark.gpu

CONFIGS = ["b256x256", "b256x128", "b128x128", "b128x128k2", "b64x128k2", "b64x64", "b64x64k2",
           "b32x128", "b32x64k4", "b32x32k4", "r16x16"]


# ------------------------------------------------------------------ routing

def run_route(x, k, bias=None, **kw):
    import torch

    import dense_gemm_bf16_amd as g

    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    ids, w = g.moe_route(x.cuda(), k, bias=b, **kw)
    return ids.cpu().numpy(), w.double().cpu().numpy()


def check_route(x, k, bias=None, **kw):
    ids, w = run_route(x, k, bias, **kw)
    want_ids, want_w = ref.route(x.float().numpy(), k, bias, **kw)
    assert np.array_equal(ids, want_ids), np.argwhere(ids != want_ids)[:4].tolist()
    # a score is off by less than 2^-18.5 relative, a sum of them by no more,
    # and the exponent x - max by one rounding of up to 104
    tol = (2.0 ** -17 + 104 * 2.0 ** -24) * np.abs(want_w) + 1e-37
    assert (np.abs(w - want_w) <= tol).all(), float(np.max(np.abs(w - want_w) / tol))


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T, E, k, groups, topk", [
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (5, 60, 4, 1, 1), (300, 64, 6, 8, 3), (17, 256, 8, 8, 4),
    (1025, 256, 8, 1, 1), (9, 160, 6, 8, 3), (7, 130, 5, 13, 6), (4, 1024, 64, 64, 33),
    (3, 1023, 9, 33, 5), (6, 1024, 16, 1, 1), (33, 12, 12, 3, 3), (8, 64, 3, 64, 3)])
def test_route(T, E, k, groups, topk, score, x_type):
    import torch

    rng = np.random.default_rng(T + E)
    x = torch.from_numpy(rng.normal(0, 1.5, (T, E))).to(dtype(x_type))
    bias = rng.normal(0, 0.2, E).astype(np.float32)
    for b in (None, bias):
        for top in (1, 2):
            for renorm in (True, False):
                check_route(x, k, b, score=score, groups=groups, topk_groups=topk, group_top=top,
                            renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest_index(score):
    import torch

    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.integers(-2, 3, (200, 96)).astype(np.float32))
    x[0] = 0
    for bias in (None, np.zeros(96), rng.integers(0, 2, 96) * 0.5):
        for groups, topk in ((1, 1), (8, 3), (3, 2)):
            for top in (1, 2):
                check_route(x, 6, bias, score=score, groups=groups, topk_groups=topk, group_top=top)


def test_route_signed_zeros_tie():
    import torch

    x = torch.zeros(2, 16)
    x[0, 0] = -0.0
    check_route(x, 3)
    check_route(x, 3, np.where(np.arange(16) % 2, 0.0, -0.0) - 0.5, score="sigmoid")


def test_route_order_is_finer_than_fp32():
    """Scores that agree to fp32's last bits: the order is that of the exact
    values.  One expert's bias makes up, to within 1e-9, for its score."""
    import torch

    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.normal(0, 1, (400, 32))).float()
    for score in ("sigmoid", "softmax"):
        s = 1 / (1 + np.exp(-x[0].double().numpy()))
        if score == "softmax":
            e = np.exp(x[0].double().numpy())
            s = e / e.sum()
        bias = (0.75 - s).astype(np.float32)  # every c of row 0 is 0.75 to fp32
        rows = x.clone()
        rows[1:] = x[0] + torch.from_numpy(rng.choice([0, 1e-7, -1e-7], (399, 32))).float()
        check_route(rows, 8, bias, score=score)
        check_route(rows, 8, bias, score=score, groups=8, topk_groups=3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E, groups, topk", [(100, 1, 1), (240, 1, 1), (240, 4, 3), (480, 1, 1),
                                             (480, 32, 9), (1000, 1, 1)])
def test_route_many_near_and_equal_scores(E, groups, topk, score):
    """One to sixteen experts a lane whose scores agree to fp32's last bits,
    or whole."""
    import torch

    rng = np.random.default_rng(E + groups)
    x = torch.from_numpy(rng.normal(0, 1, E)).float()
    e = np.exp(x.double().numpy())
    s = e / e.sum() if score == "softmax" else e / (1 + e)
    rows = x + torch.from_numpy(rng.choice([0, 1e-7, -1e-7], (60, E))).float()
    check_route(rows, 24, (0.75 - s).astype(np.float32), score=score, groups=groups,
                topk_groups=topk)
    equal = torch.from_numpy(rng.integers(0, 2, (60, E)).astype(np.float32))
    for bias in (None, np.zeros(E), rng.integers(0, 2, E) * 0.5):
        check_route(equal, 24, bias, score=score, groups=groups, topk_groups=topk)


@pytest.mark.parametrize("T, k, E", [(125, 8, 256), (300, 4, 16), (1100, 8, 5), (1600, 8, 40),
                                     (2049, 8, 9), (5000, 5, 12)])
def test_plan_parts_that_end_anywhere(T, k, E):
    """Parts of every length past whole batches of loads."""
    import torch

    import dense_gemm_bf16_amd as g

    ids = np.random.default_rng(T).integers(-1, E + 1, (T, k)).astype(np.int32)
    for a, b in zip(g.moe_plan(torch.from_numpy(ids).cuda(), E), ref.plan(ids, E)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_special_logits(score):
    import torch

    inf = float("inf")
    x = torch.randn(12, 40, generator=torch.Generator().manual_seed(1))
    x[0] = -inf                       # nothing left
    x[1, 3:] = -inf                   # fewer left than k
    x[2, 7] = inf
    x[3, [5, 9]] = inf
    x[4, 11] = float("nan")
    x[5] = float("nan")
    x[6] = torch.finfo(torch.float32).min
    x[7, ::2] = torch.finfo(torch.float32).min
    x[8] = torch.finfo(torch.float32).max
    x[9] *= 1e30
    x[10] = 88.0 + x[10]
    for bias in (None, np.linspace(-0.3, 0.3, 40)):
        for groups, topk in ((1, 1), (4, 2), (5, 5)):
            for renorm in (True, False):
                check_route(x, 5, bias, score=score, groups=groups, topk_groups=topk,
                            renormalize=renorm)
    ids, w = run_route(x, 5)
    assert (w[0] == 0).all() and sorted(ids[0]) == list(range(5))


def test_route_bias_extremes_and_strides():
    import torch

    x = torch.randn(50, 48, generator=torch.Generator().manual_seed(2))
    bias = np.zeros(48, np.float32)
    bias[5], bias[6], bias[7] = -np.inf, np.inf, np.nan
    ids, _ = run_route(x, 4, bias, score="sigmoid")
    assert (ids[:, 0] == 6).all() and not np.isin(ids, [5, 7]).any()
    wide = torch.randn(50, 51, generator=torch.Generator().manual_seed(3)).half()
    import dense_gemm_bf16_amd as g

    got, _ = g.moe_route(wide.cuda()[:, 3:], 4)  # an odd row stride, an odd start
    assert np.array_equal(got.cpu().numpy(), ref.route(wide[:, 3:].float().numpy(), 4)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [-np.inf, np.nan])
def test_masked_experts_come_last_whatever_their_bias(mask, score):
    import torch

    x = torch.full((1, 16), -0.5)
    x[0, 3] = mask
    bias = np.where(np.arange(16) == 3, 0.5, 0.0)
    ids, w = run_route(x, 2, bias, score=score)
    assert ids.tolist() == [[0, 1]] and np.abs(w - 0.5).max() <= 2.0 ** -17
    # every count of experts left, in each group and over all of them
    E = 48
    rng = np.random.default_rng(7)
    x = torch.from_numpy(rng.normal(0, 1.5, (E + 1, E))).float()
    for t in range(E + 1):
        x[t, torch.from_numpy(rng.permutation(E)[t:])] = mask
    left = x.numpy() > -np.inf  # (NaN: false)
    for bias in (np.where(left[20], -0.4, 0.6), rng.normal(0, 0.5, E)):
        for groups, topk in ((1, 1), (4, 2), (16, 5), (48, 10)):
            for top in (1, 2):
                kw = dict(score=score, groups=groups, topk_groups=topk, group_top=top)
                check_route(x, 6, bias, **kw)
                check_route(x, 6, None, **kw)
                ids, w = run_route(x, 6, bias, **kw)
                taken = np.take_along_axis(left, ids.astype(np.int64), 1)
                assert (w[~taken] == 0).all() and (w[taken] > 0).all()
                # those that are left first, and all of them where the groups do not choose
                assert (np.sort(~taken, 1) == ~taken).all()
                if topk == groups:
                    assert (taken.sum(1) == np.minimum(6, left.sum(1))).all()
                # a group with one comes before the groups without
                assert (taken[:, 0] == left.any(1)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E, groups, topk, k", [(4, 1, 1, 2), (40, 1, 1, 7), (256, 1, 1, 8), (256, 8, 3, 8),
                                                (600, 1, 1, 9), (1024, 4, 2, 30)])
def test_scores_that_are_equal_in_64_bits_go_by_logit(E, groups, topk, k, score):
    """Saturated sigmoids and softmax scores of 0: a bias of zeros, or the
    same for all, leaves the choice as it is without one."""
    import torch

    rng = np.random.default_rng(E)
    x = torch.from_numpy(rng.normal(0, 300, (30, E))).float()  # most scores are 0 or 1
    x[1] = 40 + torch.from_numpy(rng.integers(0, 4, E)).float()
    x[2] = -800 - torch.from_numpy(rng.random(E)).float()
    x[3] = torch.from_numpy(np.where(np.arange(E) % 3, 1e30, -1e30) * rng.choice([1, 2, 3], E)).float()
    x[4] = 1e-30 * x[4]
    x[5] = 37 + x[5] / 3e6  # a step or none below 1
    if E == 4:
        x[0] = torch.tensor([40.0, 50.0, 3.0, 1.0])
    kw = dict(score=score, groups=groups, topk_groups=topk)
    for top in (1, 2):
        ids, w = run_route(x, k, None, group_top=top, **kw)
        again, v = run_route(x, k, np.zeros(E), group_top=top, **kw)
        assert np.array_equal(ids, again) and np.array_equal(w, v)
        for bias in (None, np.zeros(E), rng.choice([0.0, 1.0], E)):
            assert np.array_equal(run_route(x, k, bias, group_top=top, **kw)[0],
                                  ref.route(x.numpy(), k, bias, group_top=top, **kw)[0])
    if groups == 1:
        order = np.argsort(-x.double().numpy(), axis=1, kind="stable")[:, :k]
        for bias in (0.0, 0.25, -1e9, 3e38):
            assert np.array_equal(run_route(x, k, np.full(E, bias), **kw)[0], order), bias


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E, groups, topk, k", [(8, 1, 1, 3), (64, 1, 1, 6), (256, 8, 3, 8), (1024, 1, 1, 20)])
def test_weights_of_scores_below_fp32(E, groups, topk, k, x_type):
    """Chosen scores that fp32 holds as 0, or with a few bits, have ordinary
    weights all the same: rows of logits about one level, rows across fp32's
    border, and softmax choices far below the largest logit."""
    import torch

    rng = np.random.default_rng(E)
    levels = np.array([-60.0, -69.3, -80, -87, -88.7, -89, -95, -100, -104, -300, -600, -700])
    x = levels[:, None] + rng.normal(0, 2, (len(levels), E))
    wide = -rng.uniform(40, 140, (8, E))  # chosen ones on both sides of the border
    rows = torch.from_numpy(np.concatenate([x, wide])).to(dtype(x_type))
    kw = dict(groups=groups, topk_groups=topk, scale=2.5)
    for bias in (None, rng.normal(0, 1, E)):
        check_route(rows, k, bias, score="sigmoid", **kw)
    if E == 8:
        ids, w = run_route(torch.linspace(-100, -95, 8)[None], 3, score="sigmoid")
        assert ids.tolist() == [[7, 6, 5]] and np.abs(w - [[0.578305, 0.283104, 0.138591]]).max() < 1e-5
    # one expert towers above those that the bias, or the groups, choose
    towers = rows.float()
    towers[:, 0] = towers[:, 1:].max(1).values + torch.from_numpy(rng.choice([85, 104, 110, 300, 600], len(rows)))
    towers = towers.to(dtype(x_type))
    bias = np.where(np.arange(E) == 0, -10.0, rng.normal(0, 1, E))
    for renorm in (True, False):
        check_route(towers, k, bias, renormalize=renorm, **kw)
    ids, w = run_route(towers, k, bias, **kw)
    assert (ids != 0).all() and np.abs(w.sum(1) - 2.5).max() < 1e-5


def test_a_masked_experts_row_does_not_reach_the_token():
    import torch

    import dense_gemm_bf16_amd as g

    logits = torch.zeros(3, 8, device="cuda")
    logits[:, 5] = float("-inf")
    bias = torch.zeros(8, device="cuda")
    bias[5] = 1.0
    ids, w = g.moe_route(logits, 2, bias=bias)
    offsets, rows, pos = g.moe_plan(ids, 8)
    B = torch.ones(8, 16, 64, device="cuda", dtype=torch.bfloat16)
    B[5] = float("nan")
    y = g.moe_matmul(torch.ones(3, 64, device="cuda", dtype=torch.bfloat16), B, offsets, rows=rows)
    assert bool((g.moe_combine(y, pos, w) == 64).all())


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("T, k, E", [(0, 2, 4), (1, 1, 1), (1, 8, 256), (5, 3, 7), (64, 8, 128),
                                     (512, 8, 64), (513, 8, 64), (8192, 8, 256), (3333, 7, 300)])
def test_plan(T, k, E):
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(T + E)
    for low, high in ((0, E), (-2, E + 2), (E // 2, E // 2 + 1)):
        ids = rng.integers(low, high, (T, k)).astype(np.int32)
        got = g.moe_plan(torch.from_numpy(ids).cuda(), E)
        for a, b in zip(got, ref.plan(ids, E)):
            assert np.array_equal(a.cpu().numpy(), b), (low, high)


def test_plan_of_dropped_ids_only():
    import torch

    import dense_gemm_bf16_amd as g

    ids = torch.tensor([[-1, 2 ** 31 - 1], [-2 ** 31, 4]], dtype=torch.int32).cuda()
    offsets, rows, pos = g.moe_plan(ids, 4)
    assert offsets.tolist() == [0] * 5 and rows.tolist() == [-1] * 4 and pos.tolist() == [[-1, -1]] * 2


# ------------------------------------------------------------------ experts' products

def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def experts_case(counts, T, N, K, type, seed, exact):
    import torch

    rng = np.random.default_rng(seed)
    E, R = len(counts), int(sum(counts))
    kb, nb = -(-K // 128), -(-N // 128)
    draw = (lambda s: rng.integers(-4, 5, s)) if exact else (lambda s: rng.normal(0, 1, s))
    a = torch.from_numpy(draw((T, K)).astype(np.float32)).to(dtype(type))
    b = torch.from_numpy(draw((E, N, K)).astype(np.float32)).to(dtype(type))
    sa = sb = None
    if type == "e4m3":
        scale = (lambda s: 2.0 ** rng.integers(-2, 3, s)) if exact else (lambda s: np.exp(rng.normal(-2, 1, s)))
        sa, sb = scale((kb, T)).astype(np.float32), scale((E, nb, kb)).astype(np.float32)
    rows = rng.integers(0, T, R).astype(np.int32)
    return a, b, sa, sb, rows


def run_experts(a, b, sa, sb, offsets, rows, out, config=None, c=None):
    import torch

    import dense_gemm_bf16_amd as g

    unit = 16 if sa is not None else 8
    A, B = padded(a, unit, 1), padded(b, unit, 1)
    SA = None if sa is None else padded(torch.from_numpy(sa), 1, 1)
    SB = None if sb is None else padded(torch.from_numpy(sb), 1, 2)
    got = g.moe_matmul(A, B, torch.from_numpy(offsets).cuda(),
                       rows=None if rows is None else torch.from_numpy(rows).cuda(), SA=SA, SB=SB,
                       out=c, out_dtype=None if c is not None else dtype(out), config=config)
    torch.cuda.synchronize()
    return got.float().cpu().numpy().astype(np.float64)


def want_experts(a, b, sa, sb, offsets, rows, R):
    a, b = a.float().numpy(), b.float().numpy()
    N = b.shape[1]
    C, err = np.zeros((R, N)), np.zeros((R, N))
    for e in range(b.shape[0]):
        r = rows[offsets[e]:offsets[e + 1]] if rows is not None else np.arange(offsets[e], offsets[e + 1])
        if len(r):
            C[offsets[e]:offsets[e + 1]], err[offsets[e]:offsets[e + 1]] = block_product(
                a[r], None if sa is None else sa[:, r], b[e], None if sb is None else sb[e])
    return C, err


@pytest.mark.parametrize("type", ["e4m3", "bf16", "f16"])
@pytest.mark.parametrize("config", CONFIGS)
def test_every_shape_of_experts_is_exact_on_integers(config, type):
    """Experts with no row, one, a whole tile, one more than a tile; ragged N
    and K; three output types, one rounding each."""
    import torch

    counts = [0, 1, 16, 17, 0, 65, 257, 128, 0, 3]
    a, b, sa, sb, rows = experts_case(counts, 90, 197, 328, type, 1, True)
    offsets = offsets_of(counts)
    want, _ = want_experts(a, b, sa, sb, offsets, rows, len(rows))
    for out in ("f32", "bf16", "f16"):
        got = run_experts(a, b, sa, sb, offsets, rows, out, config)
        r = torch.from_numpy(want.astype(np.float32)).to(dtype(out)).double().numpy()
        assert np.array_equal(got, r), out
    sorted_a = a[torch.from_numpy(rows).long()] if type != "e4m3" else \
        a.float()[torch.from_numpy(rows).long()].to(dtype(type))
    got = run_experts(sorted_a, b, None if sa is None else sa[:, rows], sb, offsets, None, "f32", config)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("type", ["e4m3", "bf16", "f16"])
@pytest.mark.parametrize("K", [1, 7, 8, 63, 64, 65, 127, 130, 260])
@pytest.mark.parametrize("config", ["b256x256", "b256x128", "b128x128k2", "b64x64", "b32x32k4", "r16x16"])
def test_experts_every_end_of_k(config, K, type):
    counts = [3, 0, 20]
    a, b, sa, sb, rows = experts_case(counts, 9, 33, K, type, K, True)
    want, _ = want_experts(a, b, sa, sb, offsets_of(counts), rows, 23)
    assert np.array_equal(run_experts(a, b, sa, sb, offsets_of(counts), rows, "f32", config), want)


@pytest.mark.parametrize("type", ["e4m3", "bf16", "f16"])
@pytest.mark.parametrize("counts, T, N, K", [
    ([1], 1, 256, 512), ([1] * 8, 1, 300, 1024), ([0] * 100 + [2] + [0] * 99, 2, 128, 256),
    ([5, 0, 40, 3], 30, 520, 640), ([200, 100, 0, 300], 300, 384, 512), ([600], 100, 256, 1100)])
def test_experts_automatic_shapes(counts, T, N, K, type):
    a, b, sa, sb, rows = experts_case(counts, T, N, K, type, T + N, False)
    want, err = want_experts(a, b, sa, sb, offsets_of(counts), rows, len(rows))
    for out in ("f32", "bf16"):
        check_rounded(run_experts(a, b, sa, sb, offsets_of(counts), rows, out), want, err, out)


@pytest.mark.parametrize("config", CONFIGS)
def test_rows_of_no_expert_are_left_alone(config):
    """Rows before the first expert, between and after the experts, and the
    columns beside C."""
    import torch

    offsets = np.array([5, 9, 9, 30], np.int32)
    a, b, sa, sb, rows = experts_case([4, 0, 21], 12, 45, 200, "e4m3", 2, True)
    rows = np.resize(rows, 50).astype(np.int32)
    buf = torch.full((52, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    run_experts(a, b, sa, sb, offsets, rows, "bf16", config, c=buf[1:51, 8:53])
    got = buf.float().cpu().numpy()
    want, _ = want_experts(a, b, sa, sb, offsets, rows, 50)
    r = torch.from_numpy(want.astype(np.float32)).bfloat16().float().numpy()
    assert np.array_equal(got[6:31, 8:53], r[5:30])
    got[6:31, 8:53] = 7.0
    assert (got == 7.0).all()


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("type", ["e4m3", "bf16"])
def test_rows_and_offsets_outside_are_cut(config, type):
    """A row index outside A reads as zeros; offsets past C, or running
    backwards, are cut."""
    a, b, sa, sb, rows = experts_case([10, 12], 9, 40, 136, type, 3, True)
    bad = rows.copy()
    bad[[0, 5, 21]] = [-1, 9, 2 ** 31 - 1]
    offsets = np.array([0, 10, 2 ** 30], np.int32)
    got = run_experts(a, b, sa, sb, offsets, bad, "f32", config)
    want, _ = want_experts(a, b, sa, sb, np.array([0, 10, 22]), rows, 22)
    want[[0, 5, 21]] = 0
    assert np.array_equal(got, want)
    import torch

    c = torch.full((22, 40), 7.0, device="cuda")
    run_experts(a, b, sa, sb, np.array([10, 3, -7], np.int32), rows, "f32", config, c=c)
    assert bool((c == 7.0).all())


@pytest.mark.parametrize("config", CONFIGS)
def test_overlapping_ranges_stay_inside(config):
    """Ranges that overlap give unspecified rows, but touch nothing else."""
    import torch

    a, b, sa, sb, rows = experts_case([22] * 70, 9, 40, 136, "e4m3", 3, True)
    offsets = np.tile(np.array([0, 22], np.int32), 36)[:71]
    buf = torch.full((24, 64), 7.0, device="cuda")
    run_experts(a, b, sa, sb, offsets, rows[:22], "f32", config, c=buf[1:23, 8:48])
    buf[1:23, 8:48] = 7.0
    assert bool((buf == 7.0).all())


def test_experts_without_rows_or_columns():
    import torch

    import dense_gemm_bf16_amd as g

    B = torch.zeros((3, 16, 64), device="cuda", dtype=torch.bfloat16)
    zero = torch.zeros(4, device="cuda", dtype=torch.int32)
    A = torch.zeros((0, 64), device="cuda", dtype=torch.bfloat16)
    assert g.moe_matmul(A, B, zero).shape == (0, 16)
    A = torch.ones((5, 0), device="cuda", dtype=torch.bfloat16)
    at = torch.tensor([0, 2, 5], device="cuda", dtype=torch.int32)
    C = g.moe_matmul(A, torch.ones((2, 16, 0), device="cuda", dtype=torch.bfloat16), at)
    assert bool((C == 0).all())


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("y_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T, k, N", [(1, 1, 1), (3, 2, 7), (16, 8, 4096), (100, 6, 130), (1000, 3, 520), (5, 0, 64)])
def test_combine(T, k, N, y_type, out):
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(T + N)
    R = max(1, T * k)
    y = torch.from_numpy(rng.normal(0, 1, (R, N))).to(dtype(y_type))
    pos = rng.integers(-2, R + 2, (T, k)).astype(np.int32)  # some dropped, some shared
    w = rng.random((T, k)).astype(np.float32)
    got = g.moe_combine(padded(y, 8, 1), torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(),
                        out_dtype=dtype(out)).double().cpu().numpy()
    inside = (pos >= 0) & (pos < R)
    rows = y.double().numpy()[np.where(inside, pos, 0)] * (w.astype(np.float64) * inside)[:, :, None]
    want, mag = rows.sum(1), np.abs(rows).sum(1)
    check_rounded(got, want, ref.U * (k + 1) * mag, out)


@pytest.mark.parametrize("y_type", ["bf16", "f16", "f32"])
def test_combine_rows_from_any_element(y_type):
    import torch

    import dense_gemm_bf16_amd as g

    y = torch.randn(40, 203, device="cuda").to(dtype(y_type))[:, 3:]
    pos = torch.randperm(40, device="cuda").to(torch.int32).view(10, 4)
    w = torch.rand(10, 4, device="cuda")
    for n in (199, 64, 8, 1):
        assert torch.equal(g.moe_combine(y[:, :n], pos, w), g.moe_combine(y[:, :n].contiguous(), pos, w))


def test_combine_skips_what_was_dropped():
    """A dropped slot does not touch the sum, not even as 0 * NaN."""
    import torch

    import dense_gemm_bf16_amd as g

    y = torch.full((4, 72), float("nan"), device="cuda", dtype=torch.bfloat16)
    y[1] = 2.0
    pos = torch.tensor([[1, -1], [4, 1], [-5, 100], [1, 0]], device="cuda", dtype=torch.int32)
    buf = torch.full((6, 80), 7.0, device="cuda", dtype=torch.bfloat16)
    out = g.moe_combine(y, pos, torch.full((4, 2), 0.5, device="cuda"), out=buf[1:5, :72])
    assert bool((out[:2] == 1.0).all()) and bool((out[2] == 0).all()) and bool(out[3].isnan().all())
    buf[1:5, :72] = 7.0
    assert bool((buf == 7.0).all())


# ------------------------------------------------------------------ together

def layer_inputs(T, E, H, I, seed):
    import torch

    import dense_gemm_bf16_amd as g

    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
    logits = torch.randn((T, E), device="cuda", generator=gen)
    w1 = (torch.randn((E * 2 * I, H), device="cuda", generator=gen) / H ** 0.5).bfloat16()
    w2 = (torch.randn((E * H, I), device="cuda", generator=gen) / I ** 0.5).bfloat16()
    W1, S1 = g.quantize_fp8(w1, block_rows=128)
    W2, S2 = g.quantize_fp8(w2, block_rows=128)
    return (x, logits, W1.view(E, 2 * I, H), S1.view(E, -1, S1.shape[1]), W2.view(E, H, I),
            S2.view(E, -1, S2.shape[1]))


def deq(W, S):
    W = W.double().cpu().numpy()
    S = np.repeat(np.repeat(S.double().cpu().numpy(), 128, 1), 128, 2)
    return W * S[:, :W.shape[1], :W.shape[2]]


@pytest.mark.parametrize("T", [1, 7, 200])
def test_layer(T):
    """The whole layer against 64 bits, each token by its own experts.  The
    activations are quantised twice (half an e4m3 step each, 2^-4 of a value,
    random in sign over hundreds of terms) and rounded to bf16 three times;
    a token's error stays under 6 % of its norm."""
    import torch

    import dense_gemm_bf16_amd as g

    E, H, I, k = 16, 512, 256, 4
    x, logits, W1, S1, W2, S2 = layer_inputs(T, E, H, I, 3)
    out = g.moe_mlp_fp8(x, logits, k, W1, S1, W2, S2, score="sigmoid", scale=2.0)
    ids, w = ref.route(logits.cpu().numpy(), k, score="sigmoid", scale=2.0)
    D1, D2 = deq(W1, S1), deq(W2, S2)
    X = x.double().cpu().numpy()
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            h = D1[ids[t, j]] @ X[t]
            a = h[:I] / (1 + np.exp(-h[:I])) * h[I:]
            want[t] += w[t, j] * (D2[ids[t, j]] @ a)
    got = out.double().cpu().numpy()
    off = np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)
    assert off.max() < 0.06, off.max()


def test_layer_with_dropped_pairs():
    """Experts held elsewhere: two halves of the experts, each layer dropping
    the other's pairs, add up to the whole."""
    import torch

    import dense_gemm_bf16_amd as g

    E, H, I, k = 8, 256, 128, 4
    x, logits, W1, S1, W2, S2 = layer_inputs(33, E, H, I, 4)
    ids, w = g.moe_route(logits, k)
    q, s = g.quantize_fp8(x)
    parts = []
    for e0, e1 in ((0, 8), (0, 4), (4, 8)):
        offsets, rows, pos = g.moe_plan(ids - e0, e1 - e0)
        h = g.moe_matmul(q, W1[e0:e1], offsets, rows=rows, SA=s, SB=S1[e0:e1])
        hq, hs = g.quantize_fp8(h, act="swiglu")
        y = g.moe_matmul(hq, W2[e0:e1], offsets, SA=hs, SB=S2[e0:e1], out_dtype=torch.float32)
        parts.append(g.moe_combine(y, pos, w))
    whole = parts[0].double().cpu().numpy()
    halves = (parts[1].double() + parts[2].double()).cpu().numpy()
    # the same rows in the same arithmetic: only the order of k fp32 sums differs
    mag = np.abs(whole).max()
    assert np.abs(whole - halves).max() <= 2 * k * ref.U * 8 * mag


def test_layer_in_a_graph_and_on_two_streams():
    import torch

    import dense_gemm_bf16_amd as g

    args = layer_inputs(24, 16, 512, 256, 5)
    x, logits, *weights = args
    gen = torch.Generator(device="cuda").manual_seed(6)
    run = lambda: g.moe_mlp_fp8(x, logits, 4, *weights, groups=4, topk_groups=2)  # noqa: E731
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        x.copy_(torch.randn(x.shape, device="cuda", generator=gen).bfloat16())
        logits.copy_(torch.randn(logits.shape, device="cuda", generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run()), i
    want = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for o in got:
        assert torch.equal(o, want)


def test_offsets_past_32_bits():
    """Experts 3 GB apart, rows of C and Y 126 MB apart, rows of logits and
    of what is quantised 10 GB apart: the addresses are 64-bit."""
    import torch

    import dense_gemm_bf16_amd as g

    a, b, sa, sb, rows = experts_case([20, 0, 30], 25, 130, 200, "e4m3", 8, True)
    offsets = offsets_of([20, 0, 30])
    want, _ = want_experts(a, b, sa, sb, offsets, rows, 50)
    gap = 3 << 30
    big = torch.empty(2 * gap + 130 * 208, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    B = big.as_strided((3, 130, 200), (gap, 208, 1))
    B.copy_(b.cuda())
    wide = torch.empty(50 * (30 << 20), device="cuda")
    C = wide.as_strided((50, 130), (30 << 20, 1))
    A = torch.zeros((25, 208), device="cuda").to(torch.float8_e4m3fn)[:, :200]
    A.copy_(a.cuda())
    args = [torch.from_numpy(x).cuda() for x in (offsets, rows, sa, sb)]
    for config in (None, "b256x256", "b32x128", "r16x16"):
        C.zero_()
        g.moe_matmul(A, B, args[0], rows=args[1], SA=args[2], SB=args[3], out=C, config=config)
        assert np.array_equal(C.double().cpu().numpy(), want), config
    pos = torch.arange(50, device="cuda", dtype=torch.int32).flip(0).view(25, 2)
    w = torch.rand((25, 2), device="cuda")
    assert torch.equal(g.moe_combine(C, pos, w), g.moe_combine(C.contiguous(), pos, w))
    del big, B, C
    far = torch.empty((5 << 30) + 256, device="cuda", dtype=torch.bfloat16)  # rows 5 Gi elements apart
    two = far.as_strided((2, 256), (5 << 30, 1))
    two.copy_(torch.randn((2, 256), device="cuda"))
    assert torch.equal(g.quantize_fp8(two)[1], g.quantize_fp8(two.contiguous())[1])
    assert torch.equal(g.moe_route(two, 4)[0], g.moe_route(two.contiguous(), 4)[0])
