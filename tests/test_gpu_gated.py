"""Gated products over bf16 and fp16 and the gradients of dense and gated
products, on the GPU, against 64-bit forms: bit-exact where every sum is
exact, else within bounds counted from the roundings."""
import numpy as np
import pytest

import gated_ref as ref
from block_ref import HALF_STEP, TINY, U, check_rounded, dtype, padded

pytestmark = pytest.mark.gpu

GATED = ["b256x256", "b256x192", "b256x128", "b128x128", "b128x128k2", "b64x128k2", "b64x64", "b64x64k2",
         "b32x128", "b32x64k4", "r16x16", "r16x8", "r32x16"]


def normal(rng, shape, t, sigma=1.0):
    import torch

    return torch.from_numpy(rng.normal(0, sigma, shape).astype(np.float32)).to(dtype(t))


def ints(rng, shape, t, most=3):
    import torch

    return torch.from_numpy(rng.integers(-most, most + 1, shape).astype(np.float32)).to(dtype(t))


def f64(t):
    return t.double().cpu().numpy()


def dev(t, extra=1):
    """On the GPU, rows inside a wider buffer of NaN."""
    return padded(t, 8, extra)


def forward(x, w, act="swiglu", config=None, out=None, save=True):
    import torch

    import dense_gemm_bf16_amd as g

    r = g.gated_matmul(dev(x), dev(w, 2), act=act, config=config, out=out, save=save)
    torch.cuda.synchronize()
    return r


def check_forward(h, kept, x, w, act, t):
    """h within fp32's error and one rounding of the true one; the g and u that
    were kept within it and a half step of their 24 bits."""
    F = w.shape[0] // 2
    GU, err = ref.product(f64(x), f64(w))
    g, u = GU[:, :F], GU[:, F:]
    bound = ref.gate_error(g, u, act, err[:, :F], err[:, F:])
    check_rounded(f64(h), ref.gate(g, u, act), bound, t)
    if kept is not None:
        got = ref.unkept(kept.cpu().numpy(), F)
        for v, true, e in ((got[0], g, err[:, :F]), (got[1], u, err[:, F:])):
            assert (np.abs(v - true) <= e + ref.KEPT_HALF_STEP * (np.abs(true) + e) + 2.0 ** -133).all()


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("config", GATED)
def test_gated_every_shape(config, act, t):
    """Ragged in M, F and K, padding full of NaN."""
    rng = np.random.default_rng(3)
    x, w = normal(rng, (300, 356), t), normal(rng, (2 * 197, 356), t, 356 ** -0.5)
    h, kept = forward(x, w, act, config)
    check_forward(h, kept, x, w, act, t)


@pytest.mark.parametrize("K", [0, 1, 7, 8, 9, 63, 64, 65, 127, 129, 200])
@pytest.mark.parametrize("config", GATED)
def test_gated_every_end_of_k(config, K):
    """Integers: g and u are exact, and fit what is kept of them."""
    rng = np.random.default_rng(K)
    x, w = ints(rng, (37, K), "bf16"), ints(rng, (2 * 35, K), "bf16", 2)
    h, kept = forward(x, w, "swiglu", config)
    GU = f64(x) @ f64(w).T
    assert np.abs(GU).max(initial=0) < 2 ** 12
    g, u = ref.unkept(kept.cpu().numpy(), 35)
    assert np.array_equal(np.concatenate([g, u], 1), GU)
    check_forward(h, None, x, w, "swiglu", "bf16")


@pytest.mark.parametrize("M, F, K", [
    (1, 1, 64), (1, 5000, 300), (2, 8, 8), (16, 130, 1024), (33, 1000, 640), (64, 512, 2048),
    (129, 385, 1152), (300, 640, 512), (777, 5001, 200), (1100, 4609, 136), (0, 10, 64), (5, 0, 64)])
def test_gated_automatic_shapes(M, F, K):
    rng = np.random.default_rng(M * 7 + F)
    x, w = normal(rng, (M, K), "f16"), normal(rng, (2 * F, K), "f16", K ** -0.5)
    h, kept = forward(x, w, "geglu")
    assert h.shape == (M, F) and kept.shape == (M, ref.kept_row(F))
    if M and F:
        check_forward(h, kept, x, w, "geglu", "f16")
        alone = forward(x, w, "geglu", save=False)
        assert np.array_equal(f64(alone), f64(h))  # keeping g and u changes nothing


@pytest.mark.parametrize("M, F, K", [(2507, 3315, 6400), (985, 8385, 2560), (3055, 2749, 2176)])
def test_two_launches(M, F, K):
    """Products whose last columns run in a second shape: sums of small integers
    are exact, so h, g and u are bit for bit what one shape gives."""
    import torch

    import dense_gemm_bf16_amd as g

    assert "+" in g.gated_config_name(g.GEMM_TYPE_BF16, M, F, K)
    torch.manual_seed(F)
    x = torch.randint(-3, 4, (M, K), device="cuda").bfloat16()
    w = torch.randint(-3, 4, (2 * F, K), device="cuda").bfloat16() / 64
    h, kept = g.gated_matmul(x, w, save=True)
    one, kept_one = g.gated_matmul(x, w, save=True, config="b128x128")
    assert torch.equal(h, one)
    for a, b in zip(ref.unkept(kept.cpu().numpy(), F), ref.unkept(kept_one.cpu().numpy(), F)):
        assert np.array_equal(a, b)


def test_gated_large_and_special_values():
    """Gates far out on both sides, past where the power overflows; infinities
    and NaN reach their own elements only."""
    import torch

    gates = np.array([0, -0.0, 1e-3, -1e-3, 20, -20, 87, -87, 89, -89, 200, -200, 3e4, -3e4, 1e30, -1e30],
                     np.float32)
    n = len(gates)
    x = torch.eye(n, dtype=torch.bfloat16)
    w = torch.zeros(2 * n, n, dtype=torch.bfloat16)
    w[:n] = torch.diag(torch.from_numpy(gates)).to(torch.bfloat16)
    w[n:] = 1.5
    for act in ("swiglu", "geglu"):
        h, _ = forward(x, w, act)
        g = f64(x) @ f64(w[:n]).T
        check_rounded(f64(h), ref.gate(g, np.full_like(g, 1.5), act),
                      ref.gate_error(g, np.full_like(g, 1.5), act) + 1.5 * TINY["bf16"], "bf16")
    x[3, 3], x[5, 0] = float("inf"), float("nan")
    w = torch.ones(2 * n, n, dtype=torch.bfloat16)
    h, _ = forward(x, w)
    h = f64(h)
    assert (h[3] == np.inf).all() and np.isnan(h[5]).all()
    assert np.isfinite(np.delete(h, [3, 5], 0)).all()
    h, _ = forward(x, -w)
    assert np.isnan(f64(h)[3]).all()  # -inf * 0, as g / (1 + exp(-g)) gives


@pytest.mark.parametrize("config", GATED)
def test_gated_outputs_outside_their_range_are_left_alone(config):
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(3)
    M, F, K = 70, 45, 100
    x, w = normal(rng, (M, K), "f16"), normal(rng, (2 * F, K), "f16", 0.1)
    H = torch.full((74, 64), 7.0, device="cuda", dtype=torch.float16)
    row = g.gated_kept_row(F)
    assert row == ref.kept_row(F) == 6 * 48
    kept = torch.full((74, row + 32), 99, device="cuda", dtype=torch.uint8)
    dx, dw = dev(x), dev(w)
    g.gemm_gated_ex(config, g.GEMM_TYPE_F16, M, F, K, dx, dx.stride(0), dw, dw.stride(0),
                    g.GEMM_ACT_SWIGLU, H[2:, 8:], 64, kept[1:, 16:], row + 32)
    torch.cuda.synchronize()
    check_forward(H[2:72, 8:53], kept[1:71, 16:16 + row], x, w, "swiglu", "f16")
    H[2:72, 8:53] = 7
    kept[1:71, 16:16 + row] = 99
    assert (H == 7).all() and (kept == 99).all()


def test_rows_past_32_bits():
    """An up projection that starts past 2^32 bytes into W, H past it as well."""
    import torch

    import dense_gemm_bf16_amd as g

    F, K, M = 300000, 8192, 3
    w = torch.zeros(2 * F, K, device="cuda", dtype=torch.bfloat16)
    at = [0, 1, 131071, 262144, F - 1]
    rng = np.random.default_rng(1)
    rows = normal(rng, (2 * len(at), K), "bf16", K ** -0.5).cuda()
    w[at] = rows[:len(at)]
    w[[F + i for i in at]] = rows[len(at):]
    x = normal(rng, (M, K), "bf16").cuda()
    h, kept = g.gated_matmul(x, w, save=True)
    torch.cuda.synchronize()
    check_forward(h[:, at].cpu(), None, x.cpu(), rows.cpu(), "swiglu", "bf16")
    assert int((h != 0).sum()) <= M * len(at)
    gu = f64(x) @ f64(rows).T
    for got, want in zip(ref.unkept(kept.cpu().numpy(), F), (gu[:, :len(at)], gu[:, len(at):])):
        assert np.abs(got[:, at] - want).max() < 1e-4 * np.abs(want).max()
        assert np.count_nonzero(got) <= M * len(at)
    del w, h, kept


# ------------------------------------------------------------------ gradients

SIZES = [(1, 300, 70), (300, 200, 130), (3000, 136, 72), (72, 3000, 136), (1500, 1500, 200),
         (2100, 2056, 700), (130, 4090, 8000), (4090, 130, 8000), (1030, 1030, 8000)]


def backward(dc, a, b, db_dtype=None):
    import torch

    import dense_gemm_bf16_amd as g

    r = g.matmul_backward(dev(dc), dev(a, 2), dev(b), db_dtype=db_dtype)
    torch.cuda.synchronize()
    return r


@pytest.mark.parametrize("out", [None, "f32"])
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M, N, K", [
    *SIZES, (1, 1, 1), (63, 64, 65), (257, 511, 129), (700, 1030, 520), (0, 5, 9), (5, 0, 9),
    (5, 9, 0)])
def test_product_gradients_are_exact_on_integers(M, N, K, t, out):
    """Sums of integers below 2^24 are exact in any order; padding is NaN."""
    import torch

    rng = np.random.default_rng(M + N)
    dc, a, b = (ints(rng, s, t) for s in ((M, N), (M, K), (N, K)))
    da, db = backward(dc, a, b, None if out is None else torch.float32)
    DC = f64(dc)
    wa, wb = DC @ f64(b), DC.T @ f64(a)
    assert da.shape == (M, K) and db.shape == (N, K) and da.dtype == dtype(t)
    assert np.array_equal(f64(da), torch.from_numpy(wa).float().to(dtype(t)).double().numpy())
    want = torch.from_numpy(wb).float().to(db.dtype).double().numpy()
    assert np.array_equal(f64(db), want)


def test_plans_that_the_gradients_run_as():
    """Both tiles, and splits of either product, of both and of none, are
    reached by the sizes of these tests (the others by name, above)."""
    import dense_gemm_bf16_amd as g

    seen = set()
    for M, N, K in SIZES:
        tile, x, w = g.backward_config_name(M, N, K).split("_k")
        seen.add((tile, int(x) > 1, int(w) > 1))
    one, two = False, True
    assert seen >= {("b128x128", a, b) for a in (one, two) for b in (one, two)}, seen
    assert ("b256x256", one, one) in seen, seen


@pytest.mark.parametrize("config", ["b128x128_k1_k1", "b128x128_k3_k1", "b128x128_k1_k2",
                                    "b128x128_k7_k6", "b256x256_k1_k1", "b256x256_k2_k3",
                                    "b256x256_k14_k6"])
def test_every_plan_is_exact_on_integers(config):
    """Both tiles, any split of either product, on sizes that end inside tiles,
    pieces and K-steps."""
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(5)
    M, N, K = 357, 421, 299
    dc, a, b = (ints(rng, s, "bf16") for s in ((M, N), (M, K), (N, K)))
    da, db = g.matmul_backward(dev(dc), dev(a, 2), dev(b), db_dtype=torch.float32, config=config)
    DC = f64(dc)
    assert np.array_equal(f64(db), DC.T @ f64(a))
    want = torch.from_numpy(DC @ f64(b)).float().to(torch.bfloat16).double().numpy()
    assert np.array_equal(f64(da), want)
    # a gated product's, with dG and dU that are exact: g so large that the
    # sigmoid is 1, so dg = dh u and du = dh g
    F = 213
    dh, x, w = ints(rng, (M, F), "bf16", 1), ints(rng, (M, K), "bf16"), ints(rng, (2 * F, K), "bf16", 1)
    big = rng.integers(1, 3, (M, F)) * 128.0
    u = rng.integers(-2, 3, (M, F)).astype(np.float64)
    kept = torch.from_numpy(ref.keep(big, u)).cuda()
    dx, dw = g.gated_matmul_backward(dev(dh), dev(x), dev(w, 2), kept, dw_dtype=torch.float32,
                                     config=config)
    d = np.concatenate([f64(dh) * u, f64(dh) * big], 1)
    assert np.array_equal(f64(dw), d.T @ f64(x))
    want = torch.from_numpy(d @ f64(w)).float().to(torch.bfloat16).double().numpy()
    assert np.array_equal(f64(dx), want)


@pytest.mark.parametrize("M, N, K", [(40, 5000, 100), (333, 777, 555), (1500, 100, 60), (2100, 2056, 700)])
def test_product_gradients_on_normal_values(M, N, K):
    import torch

    rng = np.random.default_rng(N)
    dc, a, b = (normal(rng, s, "bf16") for s in ((M, N), (M, K), (N, K)))
    da, db = backward(dc, a, b, torch.float32)
    want, err = ref.product(f64(dc), f64(b).T)
    check_rounded(f64(da), want, err, "bf16")
    want, err = ref.product(f64(dc).T, f64(a).T)
    check_rounded(f64(db), want, err, "f32")


def gated_backward(dh, x, w, kept, act, **kw):
    import torch

    import dense_gemm_bf16_amd as g

    r = g.gated_matmul_backward(dev(dh), dev(x), dev(w, 2), kept, act=act, **kw)
    torch.cuda.synchronize()
    return r


def check_gated_backward(dx, dw, dh, x, w, kept, act, t, w_out):
    """From the kept g and u: dg and du are off by fp32's error and a rounding
    to the type, which reach dx and dw through the products."""
    g, u = ref.unkept(kept.cpu().numpy(), dh.shape[1])
    dg, du = ref.gate_gradients(f64(dh), g, u, act)
    eg, eu = ref.gate_gradient_error(f64(dh), g, u, act)
    d, e = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    e = e + HALF_STEP[t] * (np.abs(d) + e) + TINY[t]
    W, X = f64(w), f64(x)
    k = 2 * U * (d.shape[1] + 16)
    check_rounded(f64(dx), d @ W, e @ np.abs(W) + k * ((np.abs(d) + e) @ np.abs(W)), t)
    k = 2 * U * (d.shape[0] + 16)
    check_rounded(f64(dw), d.T @ X, e.T @ np.abs(X) + k * ((np.abs(d) + e).T @ np.abs(X)), w_out)


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M, F, K", [
    (1, 1, 1), (1, 200, 64), (2, 7, 9), (65, 63, 64), (300, 197, 130), (257, 320, 72),
    (3000, 70, 40), (64, 3000, 136), (2100, 1030, 264), (130, 4090, 4090),
    (2050, 257, 8000), (8000, 130, 4090)])
def test_gated_gradients(M, F, K, t, act):
    import torch

    rng = np.random.default_rng(M + F)
    x, w = normal(rng, (M, K), t), normal(rng, (2 * F, K), t, 2 * K ** -0.5)
    dh = normal(rng, (M, F), t)
    _, kept = forward(x, w, act)
    f32 = (M + F) % 2 == 0
    dx, dw = gated_backward(dh, x, w, kept, act, dw_dtype=torch.float32 if f32 else None)
    check_gated_backward(dx, dw, dh, x, w, kept, act, t, "f32" if f32 else t)


@pytest.mark.parametrize("M, F, K", [(131072, 8, 16), (131077, 9, 24), (300001, 3, 8)])
def test_gated_gradients_of_many_rows(M, F, K):
    """More rows than the gate's gradient has workgroups for: they walk the rest."""
    import torch

    rng = np.random.default_rng(M)
    x, w, dh = normal(rng, (M, K), "bf16"), normal(rng, (2 * F, K), "bf16"), normal(rng, (M, F), "bf16")
    _, kept = forward(x, w)
    dx, dw = gated_backward(dh, x, w, kept, "swiglu", dw_dtype=torch.float32)
    check_gated_backward(dx, dw, dh, x, w, kept, "swiglu", "bf16", "f32")


def test_gated_gradients_of_more_rows_than_threads():
    """2^26 rows, each a wave's worth of the gate's gradient: 2^32 threads."""
    import torch

    import dense_gemm_bf16_amd as g

    M, F, K = (1 << 26) + 5, 8, 8
    torch.manual_seed(3)
    x = torch.randint(-300, 300, (M, K), device="cuda", dtype=torch.int16).to(torch.bfloat16) / 256
    dh = torch.randint(-300, 300, (M, F), device="cuda", dtype=torch.int16).to(torch.bfloat16) / 256
    w = torch.randn(2 * F, K, device="cuda").to(torch.bfloat16)
    h, kept = g.gated_matmul(x, w, save=True)
    dx, _ = g.gated_matmul_backward(dh, x, w, kept, dw=False)
    at = torch.cat([torch.arange(i, i + 40) for i in (0, 131052, 1 << 20, (1 << 25) - 20, M - 40)]).cuda()
    h, kept, dx, x, dh, w = h[at].cpu(), kept[at], dx[at], x[at].cpu(), dh[at].cpu(), w.cpu()
    check_forward(h, kept, x, w, "swiglu", "bf16")
    _, dw = gated_backward(dh, x, w, kept, "swiglu")
    check_gated_backward(dx, dw, dh, x, w, kept, "swiglu", "bf16", "bf16")


def test_gated_gradients_one_at_a_time_and_in_place_of_others():
    """Either output alone, and given tensors whose surroundings stay."""
    import torch

    rng = np.random.default_rng(8)
    M, F, K = 130, 77, 90
    x, w, dh = normal(rng, (M, K), "bf16"), normal(rng, (2 * F, K), "bf16", 0.1), normal(rng, (M, F), "bf16")
    _, kept = forward(x, w)
    dx, dw = gated_backward(dh, x, w, kept, "swiglu")
    only, none = gated_backward(dh, x, w, kept, "swiglu", dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = gated_backward(dh, x, w, kept, "swiglu", dx=False)
    assert none is None and torch.equal(only, dw)
    assert gated_backward(dh, x, w, kept, "swiglu", dx=False, dw=False) == (None, None)
    bx = torch.full((M + 4, 112), 7.0, device="cuda", dtype=torch.bfloat16)
    bw = torch.full((2 * F + 4, 112), 7.0, device="cuda", dtype=torch.float32)
    gated_backward(dh, x, w, kept, "swiglu", dx=bx[2:-2, 8:98], dw=bw[2:-2, 8:98])
    assert torch.equal(bx[2:-2, 8:98], dx) and torch.equal(bw[2:-2, 8:98].to(torch.bfloat16), dw)
    bx[2:-2, 8:98] = 7
    bw[2:-2, 8:98] = 7
    assert (bx == 7).all() and (bw == 7).all()


def test_the_operand_of_a_gradient_that_is_left_out_may_lie_anywhere():
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(12)
    M, F, K = 70, 40, 56
    dc, x, w = normal(rng, (M, 2 * F), "bf16"), normal(rng, (M, K), "bf16"), normal(rng, (2 * F, K), "bf16")
    dc, x, w, dh = dev(dc), dev(x), dev(w), dev(normal(rng, (M, F), "bf16"))
    _, kept = g.gated_matmul(x, w, save=True)

    def odd(t):  # the same, two bytes off 16, rows an odd number of elements apart
        wide = torch.zeros(len(t), t.shape[1] + 3, device="cuda", dtype=t.dtype)
        wide[:, 1:-2] = t
        return wide[:, 1:-2]

    pairs = ((g.matmul_backward(dc, x, odd(w), dA=False)[1], g.matmul_backward(dc, x, w, dA=False)[1]),
             (g.matmul_backward(dc, odd(x), w, dB=False)[0], g.matmul_backward(dc, x, w, dB=False)[0]),
             (g.gated_matmul_backward(dh, x, odd(w), kept, dx=False)[1],
              g.gated_matmul_backward(dh, x, w, kept, dx=False)[1]),
             (g.gated_matmul_backward(dh, odd(x), w, kept, dw=False)[0],
              g.gated_matmul_backward(dh, x, w, kept, dw=False)[0]))
    torch.cuda.synchronize()
    for got, want in pairs:
        assert torch.equal(got, want)


def test_gated_gradients_of_special_values():
    """Gates far out: nothing overflows; an infinite or NaN gradient reaches its
    own row of dx only."""
    import torch

    n = 16
    gates = torch.tensor([0, 1e-3, -1e-3, 5, -5, 50, -50, 88, -88, 150, -150, 3e4, -3e4, 1e25, -1e25, -0.0])
    gates = f64(gates.bfloat16())
    g, u = np.tile(gates, (n, 1)), np.full((n, n), 1.5)
    kept = torch.from_numpy(ref.keep(g, u)).cuda()
    x, w, dh = torch.eye(n).bfloat16(), torch.cat([torch.eye(n)] * 2).bfloat16(), torch.ones(n, n).bfloat16()
    for act in ("swiglu", "geglu"):
        dx, dw = gated_backward(dh, x, w, kept, act, dw_dtype=torch.float32)
        dg, du = ref.gate_gradients(f64(dh), g, u, act)
        eg, eu = ref.gate_gradient_error(f64(dh), g, u, act)
        tiny = 2.0 ** -126  # what the products may flush
        check_rounded(f64(dw)[:n], dg.T, (eg + HALF_STEP["bf16"] * np.abs(dg) + tiny).T, "f32")
        check_rounded(f64(dw)[n:], du.T, (eu + HALF_STEP["bf16"] * np.abs(du) + tiny).T, "f32")
    dh[3, 2], dh[7, 1] = float("inf"), float("nan")
    dx, _ = gated_backward(dh, x, w, kept, "swiglu")
    assert np.isfinite(np.delete(f64(dx), [3, 7], 0)).all()
    assert not np.isfinite(f64(dx)[3]).all() and not np.isfinite(f64(dx)[7]).all()


def test_gradients_against_differences():
    """The loss sum(r * h(x, W)) moves along a direction as the gradients say.
    (In 64 bits between the two ends; what the kernels' roundings leave is
    bounded by their outputs' norms: 2^-8 of dg, du and of the outputs, and 2^-16
    of g and u.)"""
    rng = np.random.default_rng(4)
    M, F, K = 40, 56, 48
    for act in ("swiglu", "geglu"):
        x, w = normal(rng, (M, K), "bf16"), normal(rng, (2 * F, K), "bf16", K ** -0.5)
        r = normal(rng, (M, F), "bf16")
        _, kept = forward(x, w, act)
        dx, dw = gated_backward(r, x, w, kept, act)
        X, W, R = f64(x), f64(w), f64(r)

        def loss(X, W):
            GU = X @ W.T
            return (R * ref.gate(GU[:, :F], GU[:, F:], act)).sum()

        for _ in range(4):
            ex, ew = rng.normal(0, 1, X.shape), rng.normal(0, K ** -0.5, W.shape)
            s = 1e-4
            slope = (loss(X + s * ex, W + s * ew) - loss(X - s * ex, W - s * ew)) / (2 * s)
            told = (f64(dx) * ex).sum() + (f64(dw) * ew).sum()
            size = np.linalg.norm(f64(dx)) * np.linalg.norm(ex) + np.linalg.norm(f64(dw)) * np.linalg.norm(ew)
            assert abs(slope - told) <= 3 * HALF_STEP["bf16"] * size


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["swiglu", "geglu"])
def test_each_gradient_against_differences(act, t):
    """Entries of dx and dW, one by one, against central differences of the loss
    sum(r * h(x, W)) in 64 bits.  Kept g and u are off by an fp32 sum's error and
    half a step of 24 bits, which reaches dg by |act''| <= 0.8 and |act'| <= 1.13
    (and u's likewise); dg and du are rounded once, then summed and rounded."""
    rng = np.random.default_rng(14)
    M, F, K = 40, 56, 48
    x, w = normal(rng, (M, K), t), normal(rng, (2 * F, K), t, K ** -0.5)
    r = normal(rng, (M, F), t)
    _, kept = forward(x, w, act)
    dx, dw = (f64(v) for v in gated_backward(r, x, w, kept, act))
    X, W, R = f64(x), f64(w), np.abs(f64(r))
    GU, err = ref.product(X, W)
    err = err + ref.KEPT_HALF_STEP * (np.abs(GU) + err)
    (g, u), (eg, eu) = np.split(GU, 2, 1), np.split(err, 2, 1)
    dg, du = ref.gate_gradients(f64(r), g, u, act)
    d, e = np.concatenate([dg, du], 1), np.concatenate(ref.gate_gradient_error(f64(r), g, u, act), 1)
    e = e + np.concatenate([R * (0.8 * eg * (np.abs(u) + eu) + 1.13 * eu), R * 1.13 * eg], 1)
    e = e + HALF_STEP[t] * (np.abs(d) + e) + TINY[t]
    bx = e @ np.abs(W) + 2 * U * (2 * F + 16) * ((np.abs(d) + e) @ np.abs(W))
    bw = e.T @ np.abs(X) + 2 * U * (M + 16) * ((np.abs(d) + e).T @ np.abs(X))

    def loss(X, W):
        GU = X @ W.T
        return (f64(r) * ref.gate(GU[:, :F], GU[:, F:], act)).sum()

    s = 2.0 ** -16
    for got, bound, of in ((dx, bx, X), (dw, bw, W)):
        for i in rng.choice(of.size, 400, replace=False):
            at = np.unravel_index(i, of.shape)
            one = np.zeros_like(of)
            one[at] = s
            ends = [loss(X + k * one, W) if of is X else loss(X, W + k * one) for k in (1, -1)]
            slope = (ends[0] - ends[1]) / (2 * s)
            # (the differences: a third derivative of at most 1e3 times s^2 / 6,
            # and two losses of at most 1e3 to 64 bits)
            tol = bound[at] + HALF_STEP[t] * (abs(slope) + bound[at]) + TINY[t] + 1e-7
            assert abs(got[at] - slope) <= tol, (at, got[at], slope, tol)


def test_a_captured_training_step():
    """Forward and backward in one graph, replayed with new contents between
    eager work; a second graph of other sizes beside it keeps its own
    workspace."""
    import torch

    import dense_gemm_bf16_amd as g

    def step_of(M, F, K):
        x = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
        w = torch.empty(2 * F, K, device="cuda", dtype=torch.bfloat16)
        dh = torch.empty(M, F, device="cuda", dtype=torch.bfloat16)

        def fill():
            x.normal_()
            w.normal_(0, K ** -0.5)
            dh.normal_()

        def step():
            h, kept = g.gated_matmul(x, w, save=True)
            return (h, *g.gated_matmul_backward(dh, x, w, kept))

        fill()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        return fill, step, graph, outs

    assert g.gated_backward_config_name(2048, 64, 64) != "b128x128_k1_k1"
    a, b = step_of(2048, 64, 64), step_of(600, 88, 200)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        a[0]()
        b[0]()
        torch.cuda.synchronize()
        with torch.cuda.stream(one):
            a[2].replay()
        with torch.cuda.stream(two):
            b[2].replay()
        torch.cuda.synchronize()
        for fill, step, graph, outs in (a, b):
            for p, q in zip(outs, step()):
                assert torch.equal(p, q)


# ------------------------------------------------------------------ whole layers

@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M, F, K, N", [(1, 200, 64, 72), (50, 129, 88, 101), (600, 1000, 264, 300)])
def test_a_layer_forward_and_backward(M, F, K, N, t):
    """Each of its outputs from the ones it is computed from: y and dW2 from the
    h that it returned, dx and dW1 from dh, which matmul_backward gives alone
    as the layer's backward does."""
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(M)
    x, w1, w2 = normal(rng, (M, K), t), normal(rng, (2 * F, K), t, K ** -0.5), normal(rng, (N, F), t, F ** -0.5)
    dy = normal(rng, (M, N), t)
    dx_, dw1_, dw2_, dy_ = dev(x), dev(w1), dev(w2), dev(dy)
    y, h, kept = g.gated_mlp(dx_, dw1_, dw2_, save=True)
    assert torch.equal(g.gated_mlp(dx_, dw1_, dw2_), y)
    dx, dw1, dw2 = g.gated_mlp_backward(dy_, dx_, dw1_, dw2_, h, kept, dw_dtype=torch.float32)
    dh, alone = g.matmul_backward(dy_, h, dw2_, db_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(alone, dw2)
    check_forward(h, kept, x, w1, "swiglu", t)
    want, err = ref.product(f64(h), f64(w2))
    check_rounded(f64(y), want, err, t)
    want, err = ref.product(f64(dy), f64(w2).T)
    check_rounded(f64(dh), want, err, t)
    want, err = ref.product(f64(dy).T, f64(h).T)
    check_rounded(f64(dw2), want, err, "f32")
    check_gated_backward(dx, dw1, dh.cpu(), x, w1, kept, "swiglu", t, "f32")


@pytest.mark.parametrize("M, F, K, N", [(0, 8, 9, 10), (5, 0, 9, 10), (5, 8, 0, 10), (5, 8, 9, 0),
                                        (0, 0, 0, 0)])
def test_layers_without_rows_or_columns(M, F, K, N):
    """Sums of nothing are zeros, in y and in every gradient."""
    import torch

    import dense_gemm_bf16_amd as g

    def some(*shape):
        return torch.ones(*shape, device="cuda", dtype=torch.bfloat16)

    x, w1, w2 = dev(some(M, K).cpu()), dev(some(2 * F, K).cpu()), dev(some(N, F).cpu())
    y, h, kept = g.gated_mlp(x, w1, w2, save=True)
    assert y.shape == (M, N) and h.shape == (M, F)
    if F == 0 or K == 0:
        assert (y == 0).all() and (h == 0).all()
    dx, dw1, dw2 = g.gated_mlp_backward(dev(some(M, N).cpu()), x, w1, w2, h, kept,
                                          dw_dtype=torch.float32)
    assert dx.shape == x.shape and dw1.shape == w1.shape and dw2.shape == w2.shape
    if M == 0 or N == 0:
        assert (dx == 0).all() and (dw1 == 0).all() and (dw2 == 0).all()
    q, s = g.quantize_int8(some(2 * F, K)), g.quantize_int8(some(N, F))
    y = g.gated_mlp_int8(x, *q, *s)
    assert y.shape == (M, N)
    if F == 0 or K == 0:
        assert (y == 0).all()


def test_a_layer_in_8_bit_integers():
    """Bit for bit the three operators in a row, and near the layer over the
    real weights: codes are off by half a step, 1/254 of a row's largest value,
    which for these normal values (largest about four deviations) is 1/63 of a
    deviation, uniformly: 1/110 rms, in four places (x, W1, h, W2), which the
    gate's slopes (g and u each count) at most double."""
    import torch

    import dense_gemm_bf16_amd as g

    torch.manual_seed(1)
    M, F, K, N = 70, 500, 264, 130
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    w1 = (torch.randn(2 * F, K, device="cuda") * K ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(N, F, device="cuda") * F ** -0.5).to(torch.bfloat16)
    (q1, s1), (q2, s2) = g.quantize_int8(w1), g.quantize_int8(w2)
    y = g.gated_mlp_int8(x, q1, s1, q2, s2)
    q, s = g.quantize_int8(x)
    h = g.gated_matmul_int8(q, s, q1, s1, out_dtype=torch.bfloat16)
    q, s = g.quantize_int8(h)
    assert torch.equal(y, g.matmul_int8(q, s, q2, s2, out_dtype=torch.bfloat16))
    X, A, B = f64(x), f64(w1), f64(w2)
    GU = X @ A.T
    want = ref.gate(GU[:, :F], GU[:, F:], "swiglu") @ B.T
    # h's rows reach further than four deviations: its largest value says how far
    hh = ref.gate(GU[:, :F], GU[:, F:], "swiglu")
    reach = (np.abs(hh).max(1) / np.sqrt((hh ** 2).mean(1))).max() / 4
    bound = (2 * 2 + reach + 1) / 110 + 2.0 ** -8
    assert np.linalg.norm(f64(y) - want) <= bound * np.linalg.norm(want)


def test_two_streams_at_once():
    """Layers on two streams share nothing."""
    import torch

    import dense_gemm_bf16_amd as g

    torch.manual_seed(2)
    sets, want = [], []
    for M, F, K in ((300, 704, 264), (64, 1000, 520)):
        x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
        w = (torch.randn(2 * F, K, device="cuda") * K ** -0.5).to(torch.bfloat16)
        dh = torch.randn(M, F, device="cuda").to(torch.bfloat16)
        sets.append((x, w, dh))

    def step(x, w, dh):
        h, kept = g.gated_matmul(x, w, save=True)
        return (h, *g.gated_matmul_backward(dh, x, w, kept))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M, N, K", [(256, 1024, 4096), (1, 520, 1000), (777, 1234, 600)])
def test_products_in_a_given_workspace_are_the_same(M, N, K, t):
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(M)
    a, b = dev(normal(rng, (M, K), t)), dev(normal(rng, (N, K), t))
    code = g.GEMM_TYPE_BF16 if t == "bf16" else g.GEMM_TYPE_F16
    n = g.work_size(code, M, N, K)
    ld = -(-N // 8) * 8
    c, want = (torch.full((M, ld), 7.0, device="cuda", dtype=dtype(t)) for _ in range(2))
    work = torch.full((n + 64,), 99, device="cuda", dtype=torch.uint8)
    g.gemm_work(code, M, N, K, a, a.stride(0), b, b.stride(0), c, ld, work, n)
    g.matmul(a, b, out=want[:, :N])
    torch.cuda.synchronize()
    assert torch.equal(c, want) and (work[n:] == 99).all()


@pytest.mark.parametrize("config", [None, "b128x128_k2_k3", "b256x256_k3_k2"])
def test_gradients_in_a_workspace_of_just_their_size(config):
    """Enough, and nothing past it is written."""
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(15)
    M, F, K = 300, 200, 136
    x, w, dh = (dev(normal(rng, s, "bf16")) for s in ((M, K), (2 * F, K), (M, F)))
    dc = dev(normal(rng, (M, 2 * F), "bf16"))
    _, kept = g.gated_matmul(x, w, save=True)
    wants = (g.gated_matmul_backward(dh, x, w, kept, config=config),
             g.matmul_backward(dc, x, w, config=config))
    for want, n in zip(wants, (g.gated_backward_work_size(M, F, K, config),
                               g.backward_work_size(M, 2 * F, K, config))):
        work = torch.full((n + 4096,), 99, device="cuda", dtype=torch.uint8)
        dx = torch.full((M, K), 7.0, device="cuda", dtype=torch.bfloat16)
        dw = torch.full((2 * F, K), 7.0, device="cuda", dtype=torch.bfloat16)
        outs = (dx, K, dw, K, g.GEMM_TYPE_BF16, work, n)
        if want is wants[0]:
            g.gemm_gated_backward_ex(config, g.GEMM_TYPE_BF16, M, F, K, dh, dh.stride(0), x, x.stride(0), w,
                                     w.stride(0), g.GEMM_ACT_SWIGLU, kept, kept.stride(0), *outs)
        else:
            g.gemm_backward_ex(config, g.GEMM_TYPE_BF16, M, 2 * F, K, dc, dc.stride(0), x, x.stride(0), w,
                               w.stride(0), *outs)
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and (work[n:] == 99).all()


def test_two_captured_layers_replayed_at_once():
    """Graphs captured on one stream, with split plans, replayed on two."""
    import torch

    import dense_gemm_bf16_amd as g

    torch.manual_seed(5)
    M, F, K, N = 256, 4096, 512, 1024
    assert g.work_size(g.GEMM_TYPE_BF16, M, N, F) > 0
    w1 = (torch.randn(2 * F, K, device="cuda") * K ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(N, F, device="cuda") * F ** -0.5).to(torch.bfloat16)
    xs = [torch.randn(M, K, device="cuda").to(torch.bfloat16) for _ in range(2)]
    g.gated_mlp(xs[0], w1, w2)
    torch.cuda.synchronize()
    graphs, outs, stream = [], [], torch.cuda.Stream()
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(g.gated_mlp(x, w1, w2))
        graphs.append(graph)
    sides = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        for x in xs:
            x.normal_()
        torch.cuda.synchronize()
        for graph, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(xs, outs):
            assert torch.equal(y, g.gated_mlp(x, w1, w2))


def test_gradients_past_32_bits():
    """A weight whose second half starts past 2^32 bytes, and its gradient."""
    import torch

    import dense_gemm_bf16_amd as g

    F, K, M = 300000, 8192, 3
    at = [0, 1, 131071, 262144, F - 1]
    rng = np.random.default_rng(2)
    w = torch.zeros(2 * F, K, device="cuda", dtype=torch.bfloat16)
    rows = normal(rng, (2 * len(at), K), "bf16", K ** -0.5)
    w[at], w[[F + i for i in at]] = rows[:len(at)].cuda(), rows[len(at):].cuda()
    x, dh_at = normal(rng, (M, K), "bf16"), normal(rng, (M, len(at)), "bf16")
    dh = torch.zeros(M, F, device="cuda", dtype=torch.bfloat16)
    dh[:, at] = dh_at.cuda()
    _, kept = g.gated_matmul(x.cuda(), w, save=True)
    dx, dw = g.gated_matmul_backward(dh, x.cuda(), w, kept)
    torch.cuda.synchronize()
    got = [v[:, at] for v in ref.unkept(kept.cpu().numpy(), F)]
    few = torch.from_numpy(ref.keep(*got))
    both = at + [F + i for i in at]
    check_gated_backward(dx.cpu(), dw[both].cpu(), dh_at, x, rows, few, "swiglu", "bf16", "bf16")
    assert int((dw != 0).any(1).sum()) <= 2 * len(at)
    del w, dw, dh
