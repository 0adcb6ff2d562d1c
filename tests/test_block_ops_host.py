"""The 8-bit and mixture-of-experts entry points on a machine without a GPU:
every declared function is exported and bound, and arguments that cannot be
run are refused on the host, before any device work (the pointers here are
never dereferenced)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
NUL = None
BF16, F16, F32, E4M3 = range(4)


@pytest.fixture(scope="module")
def g():
    import __graft_entry__

    b = __graft_entry__._load_builder()
    if not os.path.exists(b.LIB):
        b.build()
    import dense_gemm_bf16_amd as g

    return g


def test_declared_functions_are_exported_and_bound(g):
    text = open(os.path.join(ROOT, "include", "gemm_bf16.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_(?:fp8|moe)\w*)\s*\(", text)))
    assert names == ["gemm_fp8", "gemm_fp8_config_at", "gemm_fp8_config_name", "gemm_fp8_ex",
                     "gemm_fp8_quantize", "gemm_moe", "gemm_moe_combine", "gemm_moe_config_name",
                     "gemm_moe_ex", "gemm_moe_plan", "gemm_moe_route"]
    so = ctypes.CDLL(g.LIB_PATH)
    for n in names:
        assert hasattr(so, n) and hasattr(g, n), n


def test_config_names(g):
    names = g.fp8_config_names()
    assert len(names) == len(set(names)) >= 3
    for M in (0, 1, 16, 17, 64, 65, 300, 8192):
        for c_type in (BF16, F16, F32):
            assert all(n in names for n in g.fp8_config_name(M, 8192, 8192, c_type).split("+"))
        for type in (BF16, F16, E4M3):
            assert g.moe_config_name(type, M, 4096, 4096, 32) in names
    assert g.fp8_config_name(1, 8192, 1024) != g.fp8_config_name(8192, 8192, 1024) == "b256x256"
    assert "+" in g.fp8_config_name(777, 10240, 4104, F32)  # a part-empty last pass
    assert g.fp8_config_name(-1, 1, 1) == g.fp8_config_name(1, 1, 1, E4M3) == "invalid"
    assert g.moe_config_name(E4M3, 1, 1, 1, -1) == g.moe_config_name(F32, 1, 1, 1, 1) == "invalid"


def test_sizes_that_are_refused_have_no_shape(g):
    for M, N in ((1, 8), (300, 8192)):
        for c_type in (BF16, F16, F32):
            assert g.fp8_config_name(M, N, 131072, c_type) != "invalid"
            assert g.fp8_config_name(M, N, 131073, c_type) == "invalid"
        assert g.moe_config_name(E4M3, M, N, 131073, 4) == "invalid"
        assert g.moe_config_name(BF16, M, N, 131073, 4) != "invalid"
    assert g.fp8_config_name((1 << 31) - 1, (1 << 31) - 1, 128) == "invalid"
    assert moe(g, R=(1 << 31) - 1, N=(1 << 31) - 1, E=0, T=8, ldc=1 << 31) == 3


def test_sizes_past_the_limits_are_refused(g):
    """Before any of them enters a product that could overflow."""
    for v in (1 << 31, (1 << 63) - 16):
        ld = dict(lda=v, ldb=v, ldc=v, ldsa=v, ldsb=v)
        for M, N, K in ((v, 5, 5), (5, v, 5), (5, 5, v)):
            assert g.fp8_config_name(M, N, K) == g.moe_config_name(BF16, M, N, K, 4) == "invalid"
            assert fp8(g, M=M, N=N, K=K, **ld) == 3
            assert moe(g, type=BF16, R=M, N=N, K=K, T=M, **ld) == 3
        assert g.moe_config_name(BF16, 5, 5, 5, v) == "invalid"
        assert moe(g, E=v) == 3


def fp8(g, M=8, N=8, K=256, A=P, lda=256, SA=P, ldsa=8, B=P, ldb=256, SB=P, ldsb=2, C=P, ldc=8,
        c_type=BF16, config=None):
    return g._lib.gemm_fp8_ex(config, M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, c_type,
                              None)


@pytest.mark.parametrize("bad, code", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(lda=240), 1), (dict(ldb=240), 1),
    (dict(ldc=7), 1), (dict(ldsa=7), 1), (dict(ldsb=1), 1), (dict(A=NUL), 1), (dict(B=NUL), 1),
    (dict(C=NUL), 1), (dict(SA=NUL), 1), (dict(SB=NUL), 1), (dict(c_type=E4M3), 1),
    (dict(c_type=9), 1), (dict(A=ODD), 2), (dict(B=ODD), 2), (dict(C=ODD), 2),
    (dict(SA=ctypes.c_void_p(0x10002)), 2), (dict(lda=264), 2), (dict(ldb=264), 2),
    (dict(ldc=12), 2), (dict(config=b"nope"), 3), (dict(K=131072 + 1, lda=131088, ldb=131088,
                                                        ldsb=4000), 3),
    (dict(M=1 << 31, ldsa=1 << 31), 3), (dict(N=1 << 31, ldc=1 << 31), 3),
    (dict(ldb=1 << 28), 3), (dict(lda=1 << 28, M=300, ldsa=300, config=b"b256x256"), 3)])
def test_fp8_refusals(g, bad, code):
    assert fp8(g, **bad) == code


@pytest.mark.parametrize("config, M, N", [
    (b"b32x32k4", 65536, 65536), (b"b32x64k4", 131072, 65536), (b"r16x16", 32768, 65536),
    (b"b64x64", 1 << 20, 1 << 16), (b"b256x256", 1 << 22, 1 << 17)])
def test_grids_past_a_launch_are_refused(g, config, M, N):
    """Workgroups times their threads reach 2^32.  (Experts without any: the
    checks run, and nothing is launched.)"""
    big = dict(N=N, ldc=N, config=config)
    assert fp8(g, M=M, ldsa=M, **big) == 3
    assert moe(g, R=M, T=M, ldsa=M, rows=NUL, **big) == 3
    assert moe(g, R=M, T=M, ldsa=M, rows=NUL, E=0, **big) == 3
    assert moe(g, R=M - 256, T=M, ldsa=M, rows=NUL, E=0, **big) == 0


def test_row_strides_are_refused_only_where_no_shape_runs_them(g):
    """(Experts without any: shapes are chosen, nothing is launched.)  The
    shape that fits sizes of 8192 best loads 256 rows from one base, the
    smallest 16."""
    big = dict(R=8192, N=8192, K=4096, E=0, T=8192, lda=4096, ldsa=8192, rows=NUL, ldb=4096,
               ldsb=32, ldc=8192)
    assert g.moe_config_name(E4M3, 8192, 8192, 4096, 0) == "b256x256"
    for ld in ("lda", "ldb"):
        for stride, code in ((1 << 22, 0), (1 << 23, 0), (1 << 26, 0), ((1 << 27) - 4096, 0), (1 << 27, 3)):
            assert moe(g, **{**big, ld: stride}) == code, (ld, stride)
        assert moe(g, config=b"b256x256", **{**big, ld: 1 << 23}) == 3
        assert moe(g, config=b"b128x128", **{**big, ld: 1 << 23}) == 0
        assert moe(g, type=BF16, **{**big, ld: 1 << 25}) == 0
        assert moe(g, type=BF16, **{**big, ld: 1 << 26}) == 3
    gathered = {**big, "rows": P}
    assert moe(g, **{**gathered, "lda": 1 << 18}) == 3  # all of A from one base
    assert moe(g, **{**gathered, "lda": (1 << 18) - 16}) == 0


def test_empty_products_launch_nothing(g):
    assert fp8(g, M=0, A=NUL, SA=NUL, C=NUL) == 0
    assert fp8(g, N=0, B=NUL, SB=NUL, C=NUL) == 0
    assert moe(g, R=0, C=NUL) == 0
    assert moe(g, E=0, B=NUL, offsets=NUL) == 0
    assert quantize(g, M=0, X=NUL, Q=NUL, S=NUL) == 0
    assert quantize(g, K=0, X=NUL, Q=NUL, S=NUL) == 0
    assert route(g, T=0, X=NUL, ids=NUL, w=NUL) == 0
    assert combine(g, T=0, Y=NUL, pos=NUL, w=NUL, out=NUL) == 0
    assert combine(g, N=0, Y=NUL, pos=NUL, w=NUL, out=NUL) == 0


def moe(g, type=E4M3, R=16, N=8, K=256, E=4, T=8, A=P, lda=256, SA=P, ldsa=8, offsets=P, rows=P,
        B=P, ldb=256, sb=2048, SB=P, ldsb=2, ssb=2, C=P, ldc=8, c_type=BF16, config=None):
    return g._lib.gemm_moe_ex(config, type, R, N, K, E, T, A, lda, SA, ldsa, offsets, rows, B, ldb,
                              sb, SB, ldsb, ssb, C, ldc, c_type, None)


@pytest.mark.parametrize("bad, code", [
    (dict(R=-1), 1), (dict(E=-1), 1), (dict(T=-1), 1), (dict(type=F32), 1), (dict(type=7), 1),
    (dict(offsets=NUL), 1), (dict(rows=NUL), 1), (dict(ldsa=7), 1), (dict(sb=-16), 1),
    (dict(ssb=-1), 1), (dict(SA=NUL), 1), (dict(A=NUL), 1), (dict(sb=2040), 2),
    (dict(type=BF16, lda=260), 2), (dict(type=BF16, sb=2044), 2), (dict(offsets=ODD, config=b"x"), 3),
    (dict(offsets=ctypes.c_void_p(0x10001)), 2), (dict(rows=ctypes.c_void_p(0x10002)), 2),
    (dict(T=1 << 24, ldsa=1 << 24), 3),  # gathered rows span 2^32 bytes
    (dict(type=BF16, K=(1 << 17), lda=1 << 17, ldb=1 << 17, T=8192), 3)])
def test_moe_refusals(g, bad, code):
    assert moe(g, **bad) == code


def quantize(g, M=8, K=256, X=P, ldx=512, x_type=BF16, act=0, block=1, Q=P, ldq=256, S=P, lds=8):
    return g._lib.gemm_fp8_quantize(M, K, X, ldx, x_type, act, block, Q, ldq, S, lds, None)


@pytest.mark.parametrize("bad, code", [
    (dict(M=-1), 1), (dict(K=-1), 1), (dict(x_type=E4M3), 1), (dict(act=2), 1), (dict(block=64), 1),
    (dict(ldx=248), 1), (dict(ldx=504, act=1), 1), (dict(ldq=240), 1), (dict(lds=7), 1),
    (dict(block=128, lds=1), 1), (dict(X=NUL), 1), (dict(Q=NUL), 1), (dict(S=NUL), 1),
    (dict(X=ctypes.c_void_p(0x10001)), 2), (dict(Q=ODD), 2), (dict(ldq=264), 2),
    (dict(block=128, act=1), 3), (dict(M=1 << 31, lds=1 << 31), 3),
    (dict(block=128, M=8388481), 3)])
def test_quantize_refusals(g, bad, code):
    assert quantize(g, **bad) == code


def test_blocks_past_a_launch_are_refused(g):
    """A row of 2^24 blocks, a workgroup of 256 threads each."""
    wide = dict(block=128, ldx=1 << 31, ldq=1 << 31, lds=1 << 24)
    for K in ((1 << 31) - 127, (1 << 31) - 1):
        assert quantize(g, M=1, K=K, **wide) == 3
    assert quantize(g, M=0, K=(1 << 31) - 128, **wide) == 0


def route(g, T=4, E=64, k=8, X=P, ldx=64, x_type=F32, bias=NUL, score=0, groups=8, topk_groups=4,
          top=2, renorm=1, ids=P, w=P):
    return g._lib.gemm_moe_route(T, E, k, X, ldx, x_type, bias, score, groups, topk_groups, top,
                                 renorm, 1.0, ids, w, None)


@pytest.mark.parametrize("bad, code", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(groups=0), 1), (dict(topk_groups=0), 1),
    (dict(topk_groups=9), 1), (dict(groups=7), 1), (dict(k=33), 1), (dict(ldx=63), 1),
    (dict(score=2), 1), (dict(top=3), 1), (dict(x_type=E4M3), 1), (dict(X=NUL), 1),
    (dict(ids=NUL), 1), (dict(w=NUL), 1), (dict(X=ctypes.c_void_p(0x10002)), 2),
    (dict(E=2048, ldx=2048), 3), (dict(E=128, ldx=128, groups=128, topk_groups=64), 3),
    (dict(E=256, ldx=256, k=65, topk_groups=8), 3), (dict(T=1 << 26), 3)])
def test_route_refusals(g, bad, code):
    assert route(g, **bad) == code


@pytest.mark.parametrize("args, code", [
    ((-1, 1, 4, P, P, P, P), 1), ((4, 0, 4, P, P, P, P), 1), ((4, 1, 0, P, P, P, P), 1),
    ((4, 1, 4, NUL, P, P, P), 1), ((4, 1, 4, P, NUL, P, P), 1), ((4, 1, 4, P, P, NUL, P), 1),
    ((4, 1, 4, P, P, P, NUL), 1), ((4, 1, 4, P, ctypes.c_void_p(0x10002), P, P), 2),
    ((4, 1, 70000, P, P, P, P), 3), ((1 << 29, 4, 4, P, P, P, P), 3)])
def test_plan_refusals(g, args, code):
    assert g._lib.gemm_moe_plan(*args, None) == code


def combine(g, T=4, k=2, N=64, R=8, Y=P, ldy=64, y_type=BF16, pos=P, w=P, out=P, ldo=64, out_type=BF16):
    return g._lib.gemm_moe_combine(T, k, N, R, Y, ldy, y_type, pos, w, out, ldo, out_type, None)


@pytest.mark.parametrize("bad, code", [
    (dict(T=-1), 1), (dict(k=-1), 1), (dict(N=-1), 1), (dict(R=-1), 1), (dict(ldy=56), 1),
    (dict(ldo=56), 1), (dict(y_type=E4M3), 1), (dict(out_type=E4M3), 1), (dict(Y=NUL), 1),
    (dict(pos=NUL), 1), (dict(w=NUL), 1), (dict(out=NUL), 1), (dict(Y=ctypes.c_void_p(0x10001)), 2),
    (dict(out=ODD), 2), (dict(ldo=68), 2), (dict(T=1 << 31), 3), (dict(T=1 << 29), 3)])
def test_combine_refusals(g, bad, code):
    assert combine(g, **bad) == code


def test_tensor_forms_refuse_host_tensors(g):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, s = x.to(torch.float8_e4m3fn), torch.zeros(2, 4)
    for call in (lambda: g.quantize_fp8(x), lambda: g.matmul_fp8(q, s, q, s[:1]),
                 lambda: g.moe_route(x, 2), lambda: g.moe_plan(torch.zeros(4, 2, dtype=torch.int32), 4),
                 lambda: g.moe_matmul(x, x[None], torch.zeros(2, dtype=torch.int32)),
                 lambda: g.moe_combine(x, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_layer_refuses_logits_of_other_experts_or_tokens(g):
    """More experts than W1 holds would lose pairs, more tokens than x has
    would read zeros, without a word."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    W1, W2 = torch.zeros(8, 256, 256), torch.zeros(8, 256, 128)
    S = torch.ones(8, 2, 2)
    for T, E in ((4, 9), (4, 7), (5, 8), (3, 8)):
        with pytest.raises(ValueError, match=r"4 tokens .* 8 experts, not \(%d, %d\)" % (T, E)):
            g.moe_mlp_fp8(x, torch.zeros(T, E), 2, W1, S, W2, S[:, :, :1])
    with pytest.raises(ValueError, match="as many experts"):
        g.moe_mlp_fp8(x, torch.zeros(4, 8), 2, W1, S, W2[:7], S[:7, :, :1])
    for bad in ((x[0], torch.zeros(4, 8), W1), (x, torch.zeros(8), W1), (x, torch.zeros(4, 8), W1[0])):
        with pytest.raises(ValueError, match="need x"):
            g.moe_mlp_fp8(bad[0], bad[1], 2, bad[2], S, W2, S)
