"""Quantising rows to 8-bit integers and the products over them, on the GPU:
codes, scales and products bit for bit against the definition (sums are exact
integers; every rounding is an IEEE one), gated products within counted
bounds."""
import numpy as np
import pytest

import gated_ref as ref
from block_ref import check_rounded, dtype, padded

pytestmark = pytest.mark.gpu

CONFIGS = ["b256x256", "b256x192", "b256x128", "b128x128", "b128x128k2", "b64x128k2", "b64x64", "b64x64k2",
           "b32x128", "b32x64k4", "b32x32k4", "r16x16", "r16x8", "r32x16"]
GATED = [c for c in CONFIGS if c != "b32x32k4"]


def codes(rng, shape, lo=-128, hi=128):
    return rng.integers(lo, hi, shape).astype(np.int8)


def scales(rng, n):
    return np.exp(rng.normal(-4, 1, n)).astype(np.float32)


def wide(x, extra=1):
    """int8 codes on the GPU inside a wider buffer of 127s."""
    import torch

    return padded(torch.from_numpy(x), 16, extra, fill=127)


def product(a, sa, b, sb, out="f32", config=None, c=None):
    import torch

    import dense_gemm_bf16_amd as g

    C = g.matmul_int8(wide(a), torch.from_numpy(sa).cuda(), wide(b, 2), torch.from_numpy(sb).cuda(),
                      out=c, out_dtype=None if c is not None else dtype(out), config=config)
    torch.cuda.synchronize()
    return C.float().cpu().numpy()


def gated(a, sa, w, sw, act="swiglu", out="f32", config=None, h=None):
    import torch

    import dense_gemm_bf16_amd as g

    H = g.gated_matmul_int8(wide(a), torch.from_numpy(sa).cuda(), wide(w, 2),
                            torch.from_numpy(sw).cuda(), act=act, out=h,
                            out_dtype=None if h is not None else dtype(out), config=config)
    torch.cuda.synchronize()
    return H.double().cpu().numpy()


def rounded(x, out):
    import torch

    return torch.from_numpy(x).to(dtype(out)).float().numpy()


def check_gated(got, a, sa, w, sw, act, out):
    F = len(sw) // 2
    gu = ref.integer_product(a, sa, w, sw).astype(np.float64)
    g, u = gu[:, :F], gu[:, F:]
    check_rounded(got, ref.gate(g, u, act), ref.gate_error(g, u, act), out)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("config", CONFIGS)
def test_every_shape_bit_for_bit(config, out):
    rng = np.random.default_rng(1)
    a, b = codes(rng, (300, 712)), codes(rng, (389, 712))
    sa, sb = scales(rng, 300), scales(rng, 389) / 64
    want = rounded(ref.integer_product(a, sa, b, sb), out)
    assert np.array_equal(product(a, sa, b, sb, out, config), want)


@pytest.mark.parametrize("K", [0, 1, 15, 16, 17, 64, 100, 127, 128, 129, 143, 255, 257, 1000])
@pytest.mark.parametrize("config", CONFIGS)
def test_every_end_of_k(config, K):
    """Operands lie in buffers full of 127: what is past K must not count."""
    rng = np.random.default_rng(K)
    a, b = codes(rng, (37, K)), codes(rng, (70, K))
    sa, sb = scales(rng, 37), scales(rng, 70)
    want = ref.integer_product(a, sa, b, sb)
    assert np.array_equal(product(a, sa, b, sb, "f32", config), want)


@pytest.mark.parametrize("config", CONFIGS)
def test_largest_sums_are_exact(config):
    """-128 times -128 over all of the largest K: 2^14 x 131071 = 2^31 - 2^14,
    near the largest 32-bit integer; and alternating signs, which cancel."""
    K = 131071
    a = np.full((3, K), -128, np.int8)
    b = np.full((5, K), -128, np.int8)
    a[1, ::2], b[2] = 127, 127
    one = np.ones(5, np.float32)
    want = ref.integer_product(a, one[:3], b, one)
    assert want[0, 0] == np.float32(2 ** 31 - 2 ** 14)
    assert np.array_equal(product(a, one[:3], b, one, "f32", config), want)


@pytest.mark.parametrize("M, N, K", [
    (1, 1, 128), (1, 8192, 1024), (3, 17, 4096), (16, 130, 2048), (17, 257, 384), (33, 1000, 640),
    (64, 512, 8192), (65, 127, 256), (129, 385, 1152), (256, 640, 2048), (500, 513, 1100),
    (777, 10240, 400), (1100, 9001, 200)])
def test_automatic_shapes(M, N, K):
    rng = np.random.default_rng(M * 7 + N)
    a, b = codes(rng, (M, K)), codes(rng, (N, K))
    sa, sb = scales(rng, M), scales(rng, N) / 64
    want = ref.integer_product(a, sa, b, sb)
    for out in ("f32", "bf16"):
        assert np.array_equal(product(a, sa, b, sb, out), rounded(want, out))


@pytest.mark.parametrize("M, N, K", [(2507, 6630, 6400), (985, 16770, 2560), (3055, 5498, 2176)])
def test_two_launches(M, N, K):
    """Products whose last columns run in a second shape: bit for bit what one
    shape gives, plain and gated."""
    import torch

    import dense_gemm_bf16_amd as g

    torch.manual_seed(M)
    a = torch.randint(-128, 128, (M, K), device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (N, K), device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(M, device="cuda") / 64, torch.rand(N, device="cuda") / 64
    assert "+" in g.i8_config_name(M, N, K)
    assert "+" in g.gated_config_name(g.GEMM_TYPE_I8, M, N // 2, K)
    for t in (torch.float32, torch.bfloat16):
        c = g.matmul_int8(a, sa, b, sb, out_dtype=t)
        assert torch.equal(c, g.matmul_int8(a, sa, b, sb, out_dtype=t, config="b128x128"))
        h = g.gated_matmul_int8(a, sa, b, sb, out_dtype=t)
        assert torch.equal(h, g.gated_matmul_int8(a, sa, b, sb, out_dtype=t, config="b128x128"))


def test_special_scales():
    """Zero, infinite and NaN scales reach their own row or column only."""
    rng = np.random.default_rng(5)
    a, b = codes(rng, (40, 200), 1, 9), codes(rng, (150, 200), 1, 9)
    sa, sb = np.ones(40, np.float32), np.ones(150, np.float32)
    sa[3], sa[7], sa[9], sb[100], sb[101] = 0, np.inf, np.nan, -np.inf, 2.0 ** 127
    want = ref.integer_product(a, sa, b, sb)
    for config in CONFIGS:
        assert np.array_equal(product(a, sa, b, sb, "f32", config), want, equal_nan=True)


@pytest.mark.parametrize("config", CONFIGS)
def test_c_outside_its_range_is_left_alone(config):
    import torch

    rng = np.random.default_rng(3)
    a, b = codes(rng, (70, 200)), codes(rng, (45, 200))
    sa, sb = scales(rng, 70), scales(rng, 45)
    buf = torch.full((74, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    product(a, sa, b, sb, config=config, c=buf[2:72, 8:53])
    if config in GATED:
        product(a, sa, b, sb, config=config, c=buf[2:72, 8:53])
    got = buf.float().cpu().numpy()
    want = np.full((74, 64), 7.0, np.float32)
    want[2:72, 8:53] = rounded(ref.integer_product(a, sa, b, sb), "bf16")
    assert np.array_equal(got, want)


# ------------------------------------------------------------------ gated

@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("config", GATED)
def test_gated_every_shape(config, out, act):
    """Ragged in M, F and K; g and u are known bit for bit."""
    rng = np.random.default_rng(11)
    a, w = codes(rng, (300, 712)), codes(rng, (2 * 197, 712))
    sa, sw = scales(rng, 300) / 64, scales(rng, 394) / 8
    check_gated(gated(a, sa, w, sw, act, out, config), a, sa, w, sw, act, out)


@pytest.mark.parametrize("K", [0, 1, 15, 17, 127, 129, 143, 257])
@pytest.mark.parametrize("config", GATED)
def test_gated_every_end_of_k(config, K):
    rng = np.random.default_rng(K)
    a, w = codes(rng, (37, K)), codes(rng, (2 * 35, K))
    sa, sw = scales(rng, 37) / 8, scales(rng, 70) / 8
    check_gated(gated(a, sa, w, sw, "swiglu", "f32", config), a, sa, w, sw, "swiglu", "f32")


@pytest.mark.parametrize("M, F, K", [
    (1, 1, 128), (1, 5000, 300), (3, 17, 4096), (16, 130, 2048), (33, 1000, 640), (64, 512, 2048),
    (129, 385, 1152), (300, 640, 512), (777, 5001, 200), (1100, 4609, 200)])
def test_gated_automatic_shapes(M, F, K):
    rng = np.random.default_rng(M * 7 + F)
    a, w = codes(rng, (M, K)), codes(rng, (2 * F, K))
    sa, sw = scales(rng, M) / 64, scales(rng, 2 * F) / 8
    for out in ("f32", "f16"):
        check_gated(gated(a, sa, w, sw, "geglu", out), a, sa, w, sw, "geglu", out)


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("config", [None, *GATED])
def test_fp32_gates_are_a_few_roundings_off(config, act):
    """One product of 1 and 1 each, so g and u are the scales of their columns:
    gates over the whole range, small, far out and of every size between."""
    rng = np.random.default_rng(6)
    F = 4096
    sw = rng.normal(0, 2, 2 * F)
    sw[:1500] = rng.uniform(-9, -0.1, 1500)  # (gelu's exponent reaches 80 at -9)
    sw[1500:2500] = rng.uniform(-87, 20, 1000)
    sw[2500:3500] = rng.choice([-1, 1], 1000) * np.exp(rng.uniform(-60, 60, 1000))
    sw[3500:3512] = [0, -0.0, 88, -88, 103.9, -103.9, 200, -200, 1e30, -1e30, 3e38, -3e38]
    sw = sw.astype(np.float32)
    a, w = np.zeros((3, 40), np.int8), np.zeros((2 * F, 40), np.int8)
    a[:, 17], w[:, 17] = 1, 1
    got = gated(a, np.ones(3, np.float32), w, sw, act, "f32", config)
    g, u = sw[:F].astype(np.float64), sw[F:].astype(np.float64)
    want, bound = ref.gate(g, u, act), ref.gate_error_fp32_out(g, u, act)
    fits = np.abs(want) < np.finfo(np.float32).max
    off = np.abs(got - want)[:, fits]
    assert (off <= bound[fits]).all(), float((off / bound[fits]).max())
    assert (np.abs(got[:, ~fits]) == np.inf).all()


@pytest.mark.parametrize("config", GATED)
def test_gated_h_outside_its_range_is_left_alone(config):
    import torch

    rng = np.random.default_rng(3)
    a, w = codes(rng, (70, 200)), codes(rng, (90, 200))
    sa, sw = scales(rng, 70) / 8, scales(rng, 90) / 8
    buf = torch.full((74, 64), 7.0, device="cuda", dtype=torch.float32)
    gated(a, sa, w, sw, config=config, h=buf[2:72, 8:53])
    got = buf.double().cpu().numpy()
    check_gated(got[2:72, 8:53], a, sa, w, sw, "swiglu", "f32")
    got[2:72, 8:53] = 7
    assert (got == 7).all()


# ------------------------------------------------------------------ quantise

def quantized(x, extra=0):
    import torch

    import dense_gemm_bf16_amd as g

    q, s = g.quantize_int8(x)
    torch.cuda.synchronize()
    assert q.stride(0) % 16 == 0 and q.data_ptr() % 16 == 0
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [1, 7, 8, 9, 63, 500, 2047, 2048, 2049, 8192, 8200, 14336, 20001])
def test_quantize_bit_for_bit(K, t):
    import torch

    rng = np.random.default_rng(K)
    x = torch.from_numpy(rng.normal(0, 3, (5, K)).astype(np.float32)).to(dtype(t))
    x[1] = 0
    x[2] *= 0.001
    x[3, K // 2] = 1000.0
    q, s = quantized(x.cuda())
    want, scale = ref.quantize(x.float().numpy())
    assert np.array_equal(q, want) and np.array_equal(s, scale)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 63, 257, 4099])
def test_quantize_rows(M):
    """Rows that start at any element."""
    import torch

    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.normal(0, 1, (M, 77)).astype(np.float32)).to(dtype("bf16"))
    buf = torch.full((M, 91), float("nan"), dtype=x.dtype)
    buf[:, 3:80] = x
    q, s = quantized(buf.cuda()[:, 3:80])
    want, scale = ref.quantize(x.float().numpy())
    assert np.array_equal(q, want) and np.array_equal(s, scale)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M, K", [
    (3, 513), (3, 777), (3, 1024), (259, 1024), (259, 1025), (255, 2049), (256, 2049), (259, 4095),
    (255, 4096), (256, 4096), (259, 4097), (259, 8185), (259, 8191), (255, 8192), (256, 8192), (259, 8193)])
def test_quantize_many_rows_bit_for_bit(M, K, t):
    """Each form of the kernel for rows held in registers, at the ends of its
    columns and on both sides of the 256 rows from which four waves take a row
    of up to 8192; a row's largest value at any place of it, NaN past its end."""
    import torch

    rng = np.random.default_rng(M + K)
    v = rng.normal(0, 1, (M, K)).astype(np.float32)
    at = rng.integers(0, K, M)
    at[:9] = np.minimum([0, 7, 8, 511, 512, 2047, 2048, K - 2, K - 1], K - 1)[:M]
    v[np.arange(M), at] = rng.choice([-1, 1], M) * rng.uniform(6, 60, M)
    x = torch.from_numpy(v).to(dtype(t))
    buf = torch.full((M, K + 5), float("nan"), dtype=x.dtype)
    buf[:, 2:K + 2] = x
    for y in (buf.cuda()[:, 2:K + 2], x.cuda()):
        q, s = quantized(y)
        want, scale = ref.quantize(x.float().numpy())
        assert np.array_equal(q, want) and np.array_equal(s, scale)


def test_quantize_special_rows():
    """Largest and smallest values, ties, infinities and NaN; rows of zeros."""
    import torch

    top = float(np.finfo(np.float32).max)
    x = torch.zeros(9, 300)
    x[0, :4] = torch.tensor([top, -top, top / 2, 1.0])
    x[1, :3] = torch.tensor([2.0 ** -149, -2.0 ** -140, 2.0 ** -101])
    x[2, :5] = torch.tensor([127.0, 0.5, 1.5, -2.5, -0.5])  # ties go to even
    x[3, 250], x[3, 1], x[3, 2] = float("inf"), -float("inf"), 5.0
    x[4, 299], x[4, 0] = float("nan"), 3.0
    x[5, 0], x[5, 7], x[5, 8] = float("nan"), float("inf"), 1.0
    x[6, :] = -1.0
    x[8, 299] = 1e-30
    q, s = quantized(x.cuda())
    for r in (0, 1, 2, 6, 7, 8):
        want, scale = ref.quantize(x[r:r + 1].numpy())
        assert np.array_equal(q[r:r + 1], want) and s[r] == scale[0], r
    assert s[3] == np.inf and q[3, 250] == 127 and q[3, 1] == -127 and (np.delete(q[3], [1, 250]) == 0).all()
    assert np.isnan(s[4]) and np.isnan(s[5])


def test_quantize_rows_without_columns():
    """Scales of the floor, no codes."""
    import torch

    q, s = quantized(torch.zeros(3, 0, device="cuda", dtype=torch.bfloat16))
    assert q.shape == (3, 0) and np.array_equal(s, ref.quantize(np.zeros((3, 0)))[1])


def test_quantize_leaves_what_lies_past_k():
    import torch

    import dense_gemm_bf16_amd as g

    x = torch.randn(6, 77, device="cuda")
    q = torch.full((6, 112), 99, device="cuda", dtype=torch.int8)
    s = torch.full((8,), 5.0, device="cuda")
    g.gemm_i8_quantize(6, 77, x, 77, g.GEMM_TYPE_F32, q, 112, s)
    torch.cuda.synchronize()
    assert (q[:, 77:] == 99).all() and (s[6:] == 5).all()
    assert np.array_equal(q[:, :77].cpu().numpy(), ref.quantize(x.cpu().numpy())[0])


# ------------------------------------------------------------------ as they are used

def test_quantised_linear_layer_is_near_the_real_one():
    """x to codes, weights to codes, product: each code is off by half a step of
    its row's scale (and a product of two such errors)."""
    import torch

    import dense_gemm_bf16_amd as g

    torch.manual_seed(0)
    x = torch.randn(45, 1000, device="cuda").to(torch.bfloat16)
    w = torch.randn(333, 1000, device="cuda").to(torch.bfloat16)
    qx, sx = g.quantize_int8(x)
    qw, sw = g.quantize_int8(w)
    got = g.matmul_int8(qx, sx, qw, sw, out_dtype=torch.float32).double().cpu()
    X, W, SX, SW = x.double().cpu(), w.double().cpu(), sx.double().cpu()[:, None], sw.double().cpu()[:, None]
    hx, hw = 0.5001 * SX, 0.5001 * SW
    bound = hx @ W.abs().sum(1, keepdim=True).T + X.abs().sum(1, keepdim=True) @ hw.T + 1000 * hx @ hw.T
    assert ((got - X @ W.T).abs() <= bound + 1e-5).all()


def test_operands_on_another_stream_and_in_a_graph():
    """Captured once, replayed with new contents between eager work."""
    import torch

    import dense_gemm_bf16_amd as g

    rng = np.random.default_rng(9)
    M, F, K = 33, 100, 520
    x = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
    qw, sw = g.quantize_int8(torch.randn(2 * F, K, device="cuda"))
    side = torch.cuda.Stream()

    def layer():
        q, s = g.quantize_int8(x)
        return g.gated_matmul_int8(q, s, qw, sw), g.matmul_int8(q, s, qw, sw)

    x.normal_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer()
    for _ in range(4):
        x.copy_(torch.from_numpy(rng.normal(0, 1, (M, K)).astype(np.float32)))
        graph.replay()
        eager = layer()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)
