"""Quantising to e4m3 blocks and the products over them, on the GPU, against
64-bit forms: bit-exact where every sum is exact, else within bounds counted
from the roundings."""
import numpy as np
import pytest

from block_ref import HALF_STEP, block_product, check_rounded, cut_bound, dtype, padded

pytestmark = pytest.mark.gpu

CONFIGS = ["b256x256", "b256x128", "b128x128", "b128x128k2", "b64x128k2", "b64x64", "b64x64k2",
           "b32x128", "b32x64k4", "b32x32k4", "r16x16"]


def small_ints(rng, shape):
    return rng.integers(-4, 5, shape).astype(np.float32)


def two_powers(rng, shape):
    return 2.0 ** rng.integers(-2, 3, shape).astype(np.float32)


def product(a, sa, b, sb, out, config=None, extra=1, c=None):
    """The GPU's C; operands sit in wider buffers filled with NaN."""
    import torch

    import dense_gemm_bf16_amd as g

    A = padded(torch.from_numpy(a).to(dtype("e4m3")), 16, extra)
    B = padded(torch.from_numpy(b).to(dtype("e4m3")), 16, extra)
    SA = padded(torch.from_numpy(sa), 1, extra)
    SB = padded(torch.from_numpy(sb), 1, extra)
    C = g.matmul_fp8(A, SA, B, SB, out=c, out_dtype=None if c is not None else dtype(out),
                     config=config)
    torch.cuda.synchronize()
    return C.float().cpu().numpy().astype(np.float64)


def exact_case(M, N, K, seed):
    rng = np.random.default_rng(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    return (small_ints(rng, (M, K)), two_powers(rng, (kb, M)), small_ints(rng, (N, K)),
            two_powers(rng, (nb, kb)))


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("config", CONFIGS)
def test_every_shape_is_exact_on_integers(config, out):
    """Ragged in M, N and K; products of integers and powers of two sum
    exactly in fp32 in any order, so C is one rounding of the true sum."""
    import torch

    from dense_gemm_bf16_amd import fp8_config_names

    assert sorted(fp8_config_names()) == sorted(CONFIGS)
    a, sa, b, sb = exact_case(300, 389, 712, 1)
    got = product(a, sa, b, sb, out, config)
    want, _ = block_product(a, sa, b, sb)
    assert np.array_equal(want, want.astype(np.float32))
    ref = torch.from_numpy(want.astype(np.float32)).to(dtype(out)).float().numpy()
    assert np.array_equal(got, ref.astype(np.float64))


@pytest.mark.parametrize("K", [1, 15, 16, 17, 64, 100, 127, 128, 129, 143, 255, 257, 1000])
@pytest.mark.parametrize("config", CONFIGS)
def test_every_end_of_k(config, K):
    a, sa, b, sb = exact_case(37, 70, K, K)
    want, _ = block_product(a, sa, b, sb)
    assert np.array_equal(product(a, sa, b, sb, "f32", config), want)


@pytest.mark.parametrize("M, N, K", [
    (1, 1, 128), (1, 8192, 1024), (3, 17, 4096), (16, 130, 2048), (17, 257, 384), (33, 1000, 640),
    (64, 512, 8192), (65, 127, 256), (129, 385, 1152), (256, 640, 2048), (500, 513, 1100)])
def test_automatic_shapes_on_normal_values(M, N, K):
    import torch

    rng = np.random.default_rng(M * 7 + N)
    kb, nb = -(-K // 128), -(-N // 128)
    a = torch.from_numpy(rng.normal(0, 100, (M, K)).clip(-448, 448)).to(dtype("e4m3")).float().numpy()
    b = torch.from_numpy(rng.normal(0, 100, (N, K)).clip(-448, 448)).to(dtype("e4m3")).float().numpy()
    sa = np.exp(rng.normal(-5, 1, (kb, M))).astype(np.float32)
    sb = np.exp(rng.normal(-7, 1, (nb, kb))).astype(np.float32)
    want, err = block_product(a, sa, b, sb)
    for out in ("f32", "bf16", "f16"):
        check_rounded(product(a, sa, b, sb, out), want, err, out)


@pytest.mark.parametrize("M, N, K, out", [(260, 10000, 300, "f32"), (777, 10240, 400, "f32"),
                                          (650, 14336, 256, "bf16"), (1100, 9001, 1000, "f16")])
def test_two_launches_cover_c(M, N, K, out):
    """Products whose columns go to two shapes, on integers: every element of
    C once, with its own columns' scales.  (f16: sums stay below 65504.)"""
    import torch

    a, sa, b, sb = exact_case(M, N, K, M)
    sa /= 16
    want, _ = block_product(a, sa, b, sb)
    got = product(a, sa, b, sb, out)
    assert np.array_equal(got, torch.from_numpy(want.astype(np.float32)).to(dtype(out)).double().numpy())


def test_two_launch_plans_are_reached():
    import dense_gemm_bf16_amd as g

    codes = {"bf16": g.GEMM_TYPE_BF16, "f16": g.GEMM_TYPE_F16, "f32": g.GEMM_TYPE_F32}
    plans = [g.fp8_config_name(M, N, K, codes[o]) for M, N, K, o in
             [(260, 10000, 300, "f32"), (777, 10240, 400, "f32"), (650, 14336, 256, "bf16"),
              (1100, 9001, 1000, "f16")]]
    assert any("+" in p for p in plans), plans


def test_special_codes_and_scales():
    """Every finite e4m3 code, large scales, zero scales; a NaN code or scale
    reaches only the sums it enters.  (Codes from 256 = 2^8 on, times 2^120,
    pass fp32's largest value, just below 2^128: infinity.)"""
    import torch

    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    codes = np.where(np.isnan(codes), 0, codes)
    a = np.tile(codes, (3, 1)).astype(np.float32)
    b = np.eye(256, dtype=np.float32)
    sa = np.array([[1, 2.0 ** 60, 0], [1, 2.0 ** 60, 0]], np.float32)
    sb = np.full((2, 2), 2.0 ** 60, np.float32)
    for config in CONFIGS:
        got = product(a, sa, b, sb, "f32", config)
        want = codes[None].astype(np.float64) * np.array([[2.0 ** 60], [2.0 ** 120], [0]])
        want[want >= 2.0 ** 128], want[want <= -2.0 ** 128] = np.inf, -np.inf
        assert np.array_equal(got, want)
        a2 = a.copy()
        a2[1, 5] = np.nan
        s2 = sb.copy()
        s2[1, 1] = np.nan
        got = product(a2, sa, b, s2, "f32", config)
        assert np.isnan(got[:, 128:]).all() and np.isnan(got[1]).all()
        assert np.isfinite(got[[0, 2], :128]).all()


def test_infinite_scale_stays_in_its_columns_and_signs():
    """Three K-steps, which leaves wave groups that share K steps past the
    last one: an infinite scale of the first block gives infinities, not NaN."""
    for config in CONFIGS:
        a, b = np.ones((40, 384), np.float32), np.ones((200, 384), np.float32)
        a[3] = -1
        sb = np.ones((2, 3), np.float32)
        sb[0, 0] = np.inf
        got = product(a, np.ones((3, 40), np.float32), b, sb, "f32", config)
        want = np.full((40, 200), 384.0)
        want[:, :128] = np.inf
        want[3] *= -1
        assert np.array_equal(got, want), config


def test_c_outside_its_range_is_left_alone():
    import torch

    for config in CONFIGS:
        a, sa, b, sb = exact_case(70, 45, 200, 3)
        buf = torch.full((74, 64), 7.0, device="cuda", dtype=torch.bfloat16)
        product(a, sa, b, sb, "bf16", config, c=buf[2:72, 8:53])
        got = buf.float().cpu().numpy()
        want, _ = block_product(a, sa, b, sb)
        ref = torch.from_numpy(want.astype(np.float32)).bfloat16().float().numpy()
        assert np.array_equal(got[2:72, 8:53], ref)
        got[2:72, 8:53] = 7.0
        assert (got == 7.0).all()


def test_k_zero_gives_zeros_and_empty_shapes():
    import torch

    import dense_gemm_bf16_amd as g

    e = torch.empty((5, 0), device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.empty((0, 5), device="cuda")
    for config in CONFIGS:
        C = g.matmul_fp8(e, s, e, torch.empty((1, 0), device="cuda"), config=config)
        assert C.shape == (5, 5) and bool((C == 0).all())
    A = torch.zeros((0, 256), device="cuda", dtype=torch.float8_e4m3fn)
    B = torch.zeros((8, 256), device="cuda", dtype=torch.float8_e4m3fn)
    assert g.matmul_fp8(A, torch.empty((2, 0), device="cuda"), B, torch.ones((1, 2), device="cuda")).shape == (0, 8)


def test_repeats_are_the_same_bits():
    import torch

    import dense_gemm_bf16_amd as g

    rng = torch.Generator(device="cuda").manual_seed(1)
    for M, N, K in ((8, 4096, 4096), (300, 1000, 2000), (1024, 2048, 1024)):
        A = torch.randn((M, K), device="cuda", generator=rng).to(torch.float8_e4m3fn)
        B = torch.randn((N, K), device="cuda", generator=rng).to(torch.float8_e4m3fn)
        kb = -(-K // 128)
        SA = torch.rand((kb, M), device="cuda", generator=rng)
        SB = torch.rand((-(-N // 128), kb), device="cuda", generator=rng)
        first = g.matmul_fp8(A, SA, B, SB, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(first, g.matmul_fp8(A, SA, B, SB, out_dtype=torch.float32))


# ------------------------------------------------------------------ quantising

def quantize_ref(x):
    """Codes (as values) and scales of rows, in fp32 as the header states."""
    import torch

    M, K = x.shape
    kb = -(-K // 128)
    p = np.zeros((M, kb * 128), np.float32)
    p[:, :K] = x
    p = p.reshape(M, kb, 128)
    with np.errstate(all="ignore"):
        amax = np.fmax(np.fmax.reduce(np.abs(p), 2), np.float32(2.0 ** -100))
        inv = (np.float32(448) / amax).astype(np.float32)
        q = (p * inv[:, :, None]).reshape(M, -1)[:, :K]
        S = (amax / np.float32(448)).T
    return torch.from_numpy(q).to(torch.float8_e4m3fn).float().numpy(), S


@pytest.mark.parametrize("x_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M, K", [(1, 1), (1, 128), (3, 7), (5, 129), (16, 512), (17, 1000), (64, 2048),
                                  (130, 640), (3001, 4100)])
def test_quantize_rows_bits(M, K, x_type):
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(M + K)
    x = torch.from_numpy(rng.normal(0, 1, (M, K)) * np.exp(rng.normal(0, 3, (M, 1)))).to(dtype(x_type))
    q, S = g.quantize_fp8(padded(x, 8, 1))
    want, scale = quantize_ref(x.float().numpy())
    assert q.shape == (M, K) and S.shape == (-(-K // 128), M)
    assert np.array_equal(S.cpu().numpy(), scale)
    # (rows of the largest factor overflow fp16: infinities, so NaN codes)
    assert np.array_equal(q.float().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("x_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M, K", [(1, 1), (128, 128), (129, 100), (300, 1000), (1024, 512)])
def test_quantize_blocks_bits(M, K, x_type):
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(M + K)
    x = torch.from_numpy(rng.normal(0, 1, (M, K))).to(dtype(x_type))
    q, S = g.quantize_fp8(padded(x, 8, 1), block_rows=128)
    assert S.shape == (-(-M // 128), -(-K // 128))
    for i in range(S.shape[0]):
        part = x[128 * i:128 * i + 128].float().numpy()
        rows = part.shape[0]
        for b in range(S.shape[1]):
            block = part[:, 128 * b:128 * b + 128]
            amax = np.maximum(np.abs(block).max(), np.float32(2.0 ** -100))
            assert S[i, b].item() == amax / np.float32(448)
            want = torch.from_numpy(block * (np.float32(448) / amax)).to(torch.float8_e4m3fn)
            got = q[128 * i:128 * i + rows, 128 * b:128 * b + block.shape[1]]
            assert np.array_equal(got.float().cpu().numpy(), want.float().numpy())


@pytest.mark.parametrize("x_type", ["bf16", "f16", "f32"])
def test_quantize_rows_from_any_element(x_type):
    """Odd strides, odd starts, and an odd second half."""
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(9)
    wide = torch.from_numpy(rng.normal(0, 1, (37, 603))).to(dtype(x_type))
    x = wide.cuda()[:, 3:]
    for rows in (1, 128):
        q, S = g.quantize_fp8(x[:, :333], block_rows=rows)
        r, s = g.quantize_fp8(x[:, :333].contiguous(), block_rows=rows)
        assert torch.equal(S, s) and torch.equal(q.view(torch.uint8), r.view(torch.uint8))
    want, scale = quantize_ref(wide[:, 3:].float().numpy())
    q, S = g.quantize_fp8(x)
    assert np.array_equal(q.float().cpu().numpy(), want) and np.array_equal(S.cpu().numpy(), scale)
    a = g.quantize_fp8(x[:, :598], act="swiglu")  # 299 columns each
    b = g.quantize_fp8(torch.cat([x[:, :299], x[:, :5], x[:, 299:598], x[:, :5]], 1), act="swiglu")
    assert torch.equal(a[0][:, :256].float(), b[0][:, :256].float()) and torch.equal(a[1][:2], b[1][:2])


def test_quantize_many_rows():
    """More rows than a grid's second dimension holds workgroups of four."""
    import torch

    import dense_gemm_bf16_amd as g

    x = torch.randn((300001, 130), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    q, S = g.quantize_fp8(x)
    at = torch.tensor([0, 5, 262143, 262144, 299999, 300000], device="cuda")
    r, T = g.quantize_fp8(x[at])
    assert torch.equal(S[:, at], T)
    assert torch.equal(q.view(torch.uint8)[at], r.view(torch.uint8))


def test_quantize_special_values():
    import torch

    import dense_gemm_bf16_amd as g

    x = torch.randn(8, 256)
    x[0] = 0
    x[1] = 1e-38
    x[2, 3] = float("nan")
    x[3, 200] = float("inf")
    x[4, 128:] = 0
    x[5] = 3.4e38
    x[6, 0] = 2.0 ** -110
    x[7] = torch.finfo(torch.float32).tiny / 4
    q, S = g.quantize_fp8(x.cuda())
    want, scale = quantize_ref(x.numpy())
    assert np.array_equal(S.cpu().numpy(), scale)
    assert np.array_equal(q.float().cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want[2]).sum() == 1 and np.isnan(want[3]).sum() == 1
    assert (want[0] == 0).all() and np.isinf(scale[1, 3])


@pytest.mark.parametrize("x_type", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M, K", [(1, 8), (5, 100), (64, 2048), (1025, 4096)])
def test_quantize_swiglu(M, K, x_type):
    """Each code times its scale is within half an e4m3 step of the 64-bit
    value (a subnormal step, 2^-9 of the scale, at least).  fp32 adds: expf
    and the divisions and products, under 8 steps of 2^-23 relative; the same
    in the scale."""
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(M + K)
    x = torch.from_numpy(rng.normal(0, 2, (M, 2 * K))).to(dtype(x_type))
    q, S = g.quantize_fp8(padded(x, 8, 1), act="swiglu")
    v = x.double().numpy()
    want = v[:, :K] / (1 + np.exp(-v[:, :K])) * v[:, K:]
    scale = np.repeat(S.double().cpu().numpy().T, 128, 1)[:, :K]
    got = q.double().cpu().numpy() * scale
    slack = 8 * 2.0 ** -23
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * scale + slack * scale * 448).all()
    for b in range(S.shape[0]):
        amax = np.maximum(np.abs(want[:, 128 * b:128 * b + 128]).max(1), 2.0 ** -100)
        assert (np.abs(S[b].double().cpu().numpy() - amax / 448) <= slack * amax / 448).all()


def test_quantize_leaves_padding_alone():
    import torch

    import dense_gemm_bf16_amd as g

    x = torch.randn(20, 130, device="cuda")
    wide = torch.randn(20, 136, device="cuda")
    wide[:, :130] = x
    q = torch.full((20, 160), 3, device="cuda", dtype=torch.uint8)
    S = torch.full((3, 24), -1.0, device="cuda")
    g.gemm_fp8_quantize(20, 130, wide, 136, g.GEMM_TYPE_F32, g.GEMM_ACT_NONE, 1, q, 160, S, 24)
    want, scale = quantize_ref(x.cpu().numpy())
    assert np.array_equal(q.view(torch.float8_e4m3fn).float().cpu().numpy()[:, :130], want)
    assert bool((q[:, 130:] == 3).all())
    assert np.array_equal(S.cpu().numpy()[:2, :20], scale)
    assert bool((S[2] == -1).all()) and bool((S[:, 20:] == -1).all())


@pytest.mark.parametrize("M, N, K", [(4, 512, 1024), (300, 640, 520)])
def test_quantised_product_is_near_the_unquantised(M, N, K):
    """quantize_fp8 of both operands into matmul_fp8, against the product of
    the dequantised codes in 64 bits."""
    import torch

    import dense_gemm_bf16_amd as g

    rng = torch.Generator().manual_seed(3)
    x, w = torch.randn((M, K), generator=rng), torch.randn((N, K), generator=rng) / K ** 0.5
    q, s = g.quantize_fp8(x.to(torch.bfloat16).cuda())
    qw, sw = g.quantize_fp8(w.to(torch.bfloat16).cuda(), block_rows=128)
    got = g.matmul_fp8(q, s, qw, sw, out_dtype=torch.float32).double().cpu().numpy()
    want, err = block_product(q.float().cpu().numpy(), s.cpu().numpy(), qw.float().cpu().numpy(),
                              sw.cpu().numpy())
    check_rounded(got, want, err, "f32")
    # a code is at most half an e4m3 step off: 2^-4 of each factor, to first order
    mag = np.abs(x.bfloat16().double().numpy()) @ np.abs(w.bfloat16().double().numpy()).T
    true = x.bfloat16().double().numpy() @ w.bfloat16().double().numpy().T
    assert (np.abs(got - true) <= 0.15 * mag).all()


def test_other_stream_and_graph():
    """A captured product replayed on new inputs, eager work between."""
    import torch

    import dense_gemm_bf16_amd as g

    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((96, 1024), device="cuda", generator=gen).bfloat16()
    w = torch.randn((768, 1024), device="cuda", generator=gen).bfloat16()
    qw, sw = g.quantize_fp8(w, block_rows=128)

    def layer():
        q, s = g.quantize_fp8(x)
        return g.matmul_fp8(q, s, qw, sw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layer()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, layer())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for i in range(4):
        x.copy_(torch.randn((96, 1024), device="cuda", generator=gen).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer()), i


@pytest.mark.parametrize("M, N, K, far", [(650, 14336, 256, "A"), (40000, 256, 1024, "B")])
def test_rows_far_apart_take_a_shape_that_reaches_them(M, N, K, far):
    """Rows 8 MiB apart: 256 of them, the best shape's, span too much for one
    base, so a smaller shape runs."""
    import torch

    import dense_gemm_bf16_amd as g

    assert g.fp8_config_name(M, N, K) == "b256x256"
    rng = torch.Generator(device="cuda").manual_seed(M)
    draw = lambda n: torch.randint(-4, 5, (n, K), device="cuda", generator=rng).float().to(torch.float8_e4m3fn)  # noqa: E731
    A, B = draw(M), draw(N)
    SA = 2.0 ** torch.randint(-2, 3, (K // 128, M), device="cuda", generator=rng).float()
    SB = 2.0 ** torch.randint(-2, 3, (N // 128, K // 128), device="cuda", generator=rng).float()
    want = g.matmul_fp8(A, SA, B, SB, out_dtype=torch.float32)
    rows = M if far == "A" else N
    wide = torch.empty(rows << 23, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    apart = wide.as_strided((rows, K), (1 << 23, 1))
    apart.copy_(A if far == "A" else B)
    if far == "A":
        A = apart
    else:
        B = apart
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(g.matmul_fp8(A, SA, B, SB, out_dtype=out), want.to(out))
    with pytest.raises(g.GemmError):
        g.matmul_fp8(A, SA, B, SB, config="b256x256")


@pytest.mark.parametrize("M, N, K, out", [
    (M, N, K, out) for M, N, K in ((641, 21768, 70), (694, 24955, 272), (2869, 6675, 275),
                                   (1007, 16422, 444), (1252, 6536, 973)) for out in ("bf16", "f16")] +
    [(291, 26435, 267, "f32"), (1052, 7171, 274, "f32"), (2084, 4784, 402, "f32")])
def test_each_two_launch_plan_covers_c(M, N, K, out):
    """Each of these runs as two launches, for both 16-bit types and fp32: on
    integers every element of C once, with its own columns' scales, and
    nothing beside C.  (f16: sums stay below 65504.)"""
    import torch

    import dense_gemm_bf16_amd as g

    code = {"bf16": g.GEMM_TYPE_BF16, "f16": g.GEMM_TYPE_F16, "f32": g.GEMM_TYPE_F32}[out]
    assert "+" in g.fp8_config_name(M, N, K, code)
    a, sa, b, sb = exact_case(M, N, K, M)
    sa /= 16
    want, _ = block_product(a, sa, b, sb)
    ld = -(-N // 8) * 8 + 16
    buf = torch.full((M + 2, ld), 7.0, device="cuda", dtype=dtype(out))
    product(a, sa, b, sb, out, c=buf[1:M + 1, 8:8 + N])
    got = buf.float().cpu()
    assert torch.equal(got[1:M + 1, 8:8 + N], torch.from_numpy(want.astype(np.float32)).to(dtype(out)).float())
    got[1:M + 1, 8:8 + N] = 7.0
    assert bool((got == 7.0).all())


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("config", CONFIGS)
def test_products_that_cancel(config, out):
    """Outliers, products that cancel to nothing beside small ones, and
    subnormal codes: a 16-bit C within what the matrix instruction cuts off,
    fp32 C as if nothing were large."""
    import torch

    rng = np.random.default_rng(11)
    M, N, K = 40, 70, 400
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    codes = codes[np.isfinite(codes)]
    a, b = rng.choice(codes, (M, K)), rng.choice(codes, (N, K))  # every exponent alike
    a[8:16], b[8:16] = rng.choice([-1, 1], (8, K)), rng.choice([1, 2], (8, K))
    a[16:24] *= rng.choice([0, 1], (8, K), p=[0.9, 0.1])
    for i, (p, q) in enumerate(((0, 1), (0, 127), (5, 9), (128, 399), (130, 135), (3, 260))):
        a[8 + i, p], a[8 + i, q] = 448, -448  # sums of small products beside +-448 * 448
        b[8:16, p] = b[8:16, q] = 448
    a, b = a.astype(np.float32), b.astype(np.float32)
    kb, nb = 4, 1
    sa, sb = np.full((kb, M), 2.0 ** -5, np.float32), np.full((nb, kb), 2.0 ** -6, np.float32)
    want, err = block_product(a, sa, b, sb)
    got = product(a, sa, b, sb, out, config)
    check_rounded(got, want, err if out == "f32" else err + cut_bound(a, sa, b, sb), out)


def test_small_products_beside_a_cancelled_one():
    """Where the eights' borders lie, and that fp32 C loses nothing."""
    a, b = np.zeros((3, 128), np.float32), np.zeros((1, 128), np.float32)
    b[0, [0, 9]] = 448
    b[0, 10:127] = 1
    a[:, 10:127] = 1                  # 117 products of 1
    a[1, 0], a[1, 9] = 448, -448      # 0 .. 7 and 8 .. 15: six ones beside the second
    a[2, 0], a[2, 9] = 1, 1
    one = np.ones((1, 3), np.float32)
    for config in CONFIGS:
        got = product(a, one, b, one[:, :1], "f32", config)
        assert got.tolist() == [[117], [117], [117 + 2 * 448]]
        got = product(a, one, b, one[:, :1], "bf16", config)
        assert got[0] == 117 and 117 - 6 <= got[1] <= 117
