"""The integer, gated and gradient entry points on a machine without a GPU:
every declared function is exported and bound, and arguments that cannot be
run are refused on the host, before any device work (the pointers here are
never dereferenced)."""
import ctypes
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
NUL = None
BF16, F16, F32, E4M3, I8 = range(5)


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
    names = sorted(set(re.findall(r"\b(gemm_(?:i8|gated|backward|work)\w*)\s*\(", text)))
    assert names == ["gemm_backward", "gemm_backward_config_name", "gemm_backward_ex",
                     "gemm_backward_work_size", "gemm_gated", "gemm_gated_backward",
                     "gemm_gated_backward_config_name", "gemm_gated_backward_ex",
                     "gemm_gated_backward_work_size", "gemm_gated_config_name", "gemm_gated_ex",
                     "gemm_gated_kept_row", "gemm_i8", "gemm_i8_config_at", "gemm_i8_config_name", "gemm_i8_ex",
                     "gemm_i8_gated", "gemm_i8_gated_ex", "gemm_i8_quantize", "gemm_work",
                     "gemm_work_size"]
    so = ctypes.CDLL(g.LIB_PATH)
    for n in names:
        assert hasattr(so, n) and hasattr(g, n), n
    for n, v in (("TYPE_I8", I8), ("ACT_GEGLU", 2)):
        assert getattr(g, "GEMM_" + n) == v
        assert re.search(r"#define GEMM_%s %d\b" % (n, v), open(os.path.join(ROOT, "include", "gemm_bf16.h")).read())


def test_config_names(g):
    names = g.i8_config_names()
    assert len(names) == len(set(names)) >= 3 and g.gemm_i8_config_at(-1) is None
    for M in (0, 1, 16, 17, 64, 65, 300, 8192):
        assert all(n in names for n in g.i8_config_name(M, 8192, 8192).split("+"))
        for t in (BF16, F16, I8):
            used = g.gated_config_name(t, M, 4096, 4096).split("+")
            assert all(n in names and n != "b32x32k4" for n in used)
    assert g.i8_config_name(1, 1024, 1024) != g.i8_config_name(8192, 8192, 8192) == "b256x256"
    assert g.gated_config_name(F32, 1, 8, 8) == g.gated_config_name(E4M3, 1, 8, 8) == "invalid"
    for v in (-1, 1 << 31, (1 << 63) - 1):
        for s in ((v, 5, 5), (5, v, 5), (5, 5, v)):
            assert g.i8_config_name(*s) == g.gated_config_name(BF16, *s) == "invalid"
            assert g.backward_config_name(*s) == g.gated_backward_config_name(*s) == "invalid"
            assert g.backward_work_size(*s) == g.gated_backward_work_size(*s) == 0
    assert g.i8_config_name(5, 5, 131071) != "invalid" == g.i8_config_name(5, 5, 131072)
    assert g.gated_config_name(BF16, 5, 5, 131072) != "invalid" == g.gated_config_name(I8, 5, 5, 131072)


def i8(g, M=8, N=8, K=256, A=P, lda=256, SA=P, B=P, ldb=256, SB=P, C=P, ldc=8, c_type=BF16,
       config=None):
    return g._lib.gemm_i8_ex(config, M, N, K, A, lda, SA, B, ldb, SB, C, ldc, c_type, None)


@pytest.mark.parametrize("bad, code", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(lda=240), 1), (dict(ldb=240), 1),
    (dict(ldc=7), 1), (dict(A=NUL), 1), (dict(B=NUL), 1), (dict(C=NUL), 1), (dict(SA=NUL), 1),
    (dict(SB=NUL), 1), (dict(c_type=E4M3), 1), (dict(c_type=I8), 1), (dict(c_type=9), 1),
    (dict(A=ODD), 2), (dict(B=ODD), 2), (dict(C=ODD), 2), (dict(SA=ctypes.c_void_p(0x10002)), 2),
    (dict(SB=ctypes.c_void_p(0x10001)), 2), (dict(lda=264), 2), (dict(ldb=264), 2),
    (dict(ldc=12), 2), (dict(config=b"nope"), 3), (dict(K=131072, lda=131072, ldb=131072), 3),
    (dict(M=1 << 31), 3), (dict(N=1 << 31, ldc=1 << 31), 3), (dict(ldc=1 << 40), 3),
    (dict(ldb=1 << 29), 3), (dict(lda=1 << 28, M=300, config=b"b256x256"), 3),
    (dict(M=1 << 22, N=1 << 17, ldc=1 << 17, config=b"b256x256"), 3)])
def test_i8_refusals(g, bad, code):
    assert i8(g, **bad) == code


def i8_gated(g, M=8, F=8, K=256, A=P, lda=256, SA=P, W=P, ldw=256, SW=P, act=1, H=P, ldh=8,
             h_type=BF16, config=None):
    return g._lib.gemm_i8_gated_ex(config, M, F, K, A, lda, SA, W, ldw, SW, act, H, ldh, h_type, None)


@pytest.mark.parametrize("bad, code", [
    (dict(M=-1), 1), (dict(F=-1), 1), (dict(act=0), 1), (dict(act=3), 1), (dict(ldh=7), 1),
    (dict(SW=NUL), 1), (dict(W=NUL), 1), (dict(h_type=I8), 1), (dict(W=ODD), 2), (dict(ldw=264), 2),
    (dict(F=1 << 30, ldh=1 << 30), 3), (dict(K=131072, lda=131072, ldw=131072), 3),
    (dict(config=b"b32x32k4"), 3), (dict(config=b"x"), 3)])
def test_i8_gated_refusals(g, bad, code):
    assert i8_gated(g, **bad) == code


def gated(g, type=BF16, M=8, F=9, K=64, X=P, ldx=64, W=P, ldw=64, act=1, H=P, ldh=16, kept=P,
          ld_kept=96, config=None):
    return g._lib.gemm_gated_ex(config, type, M, F, K, X, ldx, W, ldw, act, H, ldh, kept, ld_kept,
                                None)


@pytest.mark.parametrize("bad, code", [
    (dict(type=I8), 1), (dict(type=F32), 1), (dict(type=E4M3), 1), (dict(M=-1), 1), (dict(F=-1), 1),
    (dict(K=-1), 1), (dict(act=0), 1), (dict(ldx=56), 1), (dict(ldw=56), 1), (dict(ldh=8), 1),
    (dict(ld_kept=80), 1), (dict(X=NUL), 1), (dict(W=NUL), 1), (dict(H=NUL), 1), (dict(X=ODD), 2),
    (dict(W=ODD), 2), (dict(H=ODD), 2), (dict(kept=ODD), 2), (dict(ldx=68), 2), (dict(ldw=68), 2),
    (dict(ldh=20), 2), (dict(ld_kept=104), 2), (dict(F=1 << 30, ldh=1 << 30, ld_kept=1 << 33), 3),
    (dict(K=1 << 30, ldx=1 << 30, ldw=1 << 30), 3), (dict(ldw=1 << 29), 3),
    (dict(config=b"b32x32k4"), 3)])
def test_gated_refusals(g, bad, code):
    assert gated(g, **bad) == code


def quantize(g, M=8, K=250, X=P, ldx=256, x_type=BF16, Q=P, ldq=256, S=P):
    return g._lib.gemm_i8_quantize(M, K, X, ldx, x_type, Q, ldq, S, None)


@pytest.mark.parametrize("bad, code", [
    (dict(M=-1), 1), (dict(K=-1), 1), (dict(x_type=E4M3), 1), (dict(x_type=I8), 1), (dict(ldx=249), 1),
    (dict(ldq=240), 1), (dict(X=NUL), 1), (dict(Q=NUL), 1), (dict(S=NUL), 1),
    (dict(X=ctypes.c_void_p(0x10001)), 2), (dict(x_type=F32, X=ctypes.c_void_p(0x10002)), 2),
    (dict(Q=ODD), 2), (dict(ldq=264), 2), (dict(S=ctypes.c_void_p(0x10002)), 2), (dict(M=1 << 22), 3),
    (dict(K=1 << 31, ldx=1 << 31, ldq=1 << 31), 3), (dict(ldx=1 << 40), 3)])
def test_quantize_refusals(g, bad, code):
    assert quantize(g, **bad) == code


def backward(g, type=BF16, M=8, N=16, K=64, dC=P, lddc=16, A=P, lda=64, B=P, ldb=64, dA=P, ldda=64,
             dB=P, lddb=64, db_type=BF16, work=P, nbytes=1 << 30, config=None):
    return g._lib.gemm_backward_ex(config, type, M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb,
                                db_type, work, nbytes, None)


@pytest.mark.parametrize("bad, code", [
    (dict(type=F32), 1), (dict(type=I8), 1), (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1),
    (dict(db_type=F16), 1), (dict(db_type=E4M3), 1), (dict(lddc=8), 1), (dict(lda=56), 1),
    (dict(ldb=56), 1), (dict(ldda=56), 1), (dict(lddb=56), 1), (dict(dC=NUL), 1), (dict(A=NUL), 1),
    (dict(B=NUL), 1), (dict(dC=ODD), 2), (dict(A=ODD), 2), (dict(B=ODD), 2), (dict(dA=ODD), 2),
    (dict(dB=ODD), 2), (dict(work=ODD), 2), (dict(lddc=20), 2), (dict(lda=68), 2), (dict(ldb=68), 2),
    (dict(ldda=68), 2), (dict(lddb=68), 2), (dict(M=1 << 30), 3), (dict(K=1 << 30), 3),
    (dict(N=1 << 29, lddc=1 << 29), 3), (dict(lddc=1 << 40), 3), (dict(lddc=1 << 22), 3),
    (dict(lda=1 << 24), 3), (dict(ldb=1 << 24), 3), (dict(config=b"b64x64_k1_k1"), 3),
    (dict(config=b"b128x128"), 3), (dict(config=b"b128x128_k1"), 3),
    (dict(config=b"b128x128_k0_k1"), 3), (dict(config=b"b128x128_k1_k65"), 3),
    (dict(config=b"b128x128_k1_k1x"), 3),
    (dict(M=1 << 20, N=4096, K=1 << 17, lddc=4096, lda=1 << 17, ldb=1 << 17, ldda=1 << 17,
          lddb=1 << 17, config=b"b128x128_k64_k1"), 3)])  # 2^32 threads
def test_backward_refusals(g, bad, code):
    assert backward(g, **bad) == code


def gated_backward(g, type=F16, M=8, F=9, K=64, dH=P, lddh=16, X=P, ldx=64, W=P, ldw=64, act=1,
                   kept=P, ld_kept=96, dX=P, lddx=64, dW=P, lddw=64, dw_type=F32, work=P, nbytes=1 << 30,
                   config=None):
    return g._lib.gemm_gated_backward_ex(config, type, M, F, K, dH, lddh, X, ldx, W, ldw, act, kept, ld_kept, dX,
                                      lddx, dW, lddw, dw_type, work, nbytes, None)


@pytest.mark.parametrize("bad, code", [
    (dict(type=F32), 1), (dict(type=I8), 1), (dict(M=-1), 1), (dict(F=-1), 1), (dict(K=-1), 1),
    (dict(act=0), 1), (dict(act=3), 1), (dict(dw_type=BF16), 1), (dict(lddh=8), 1), (dict(ldx=56), 1),
    (dict(ldw=56), 1), (dict(ld_kept=80), 1), (dict(lddx=56), 1), (dict(lddw=56), 1), (dict(dH=NUL), 1),
    (dict(X=NUL), 1), (dict(W=NUL), 1), (dict(kept=NUL), 1), (dict(dH=ODD), 2), (dict(kept=ODD), 2),
    (dict(dX=ODD), 2), (dict(dW=ODD), 2), (dict(work=ODD), 2), (dict(lddh=20), 2), (dict(ld_kept=104), 2),
    (dict(lddx=68), 2), (dict(lddw=68), 2), (dict(work=NUL), 6), (dict(nbytes=0), 6), (dict(M=1 << 30), 3),
    (dict(F=1 << 29, lddh=1 << 29, ld_kept=1 << 32), 3), (dict(F=(1 << 63) - 1), 3),
    (dict(M=1 << 20, F=1 << 16, lddh=1 << 16, ld_kept=1 << 19), 3), (dict(ldw=1 << 24), 3),
    (dict(F=1 << 22, lddh=1 << 22, ld_kept=1 << 25), 3), (dict(config=b"b128x128_k1"), 3)])
def test_gated_backward_refusals(g, bad, code):
    assert gated_backward(g, **bad) == code


def work(g, type=BF16, M=256, N=8192, K=8192, A=P, lda=8192, B=P, ldb=8192, C=P, ldc=8192, work=P,
         nbytes=1 << 30):
    return g._lib.gemm_work(type, M, N, K, A, lda, B, ldb, C, ldc, work, nbytes, None)


@pytest.mark.parametrize("bad, code", [
    (dict(type=F32), 1), (dict(type=I8), 1), (dict(M=-1), 1), (dict(lda=8184), 1), (dict(A=NUL), 1),
    (dict(C=NUL), 1), (dict(A=ODD), 2), (dict(work=ODD), 2), (dict(ldc=8196), 2), (dict(work=NUL), 6),
    (dict(nbytes=1 << 20), 6), (dict(M=0, C=NUL, work=NUL), 0), (dict(ldb=1 << 30), 3)])
def test_work_refusals(g, bad, code):
    assert work(g, **bad) == code


def test_work_sizes_are_the_dense_products(g):
    for M, N, K in ((1, 8192, 8192), (256, 8192, 8192), (512, 10240, 8192), (4096, 4096, 4096)):
        for t in (BF16, F16):
            assert g.work_size(t, M, N, K) == g.workspace_size(M, N, K)
    assert g.work_size(BF16, 256, 8192, 8192) > 0 == g.work_size(F32, 256, 8192, 8192)


def test_workspaces(g):
    """What the size functions say is enough, a byte less is not, and a
    gradient that is left out needs no more."""
    M, N, K = 8, 4096, 64  # split: one tile of dA, 64 steps
    need = g.backward_work_size(M, N, K)
    assert need > 0 and g.backward_config_name(M, N, K) != "b128x128_k1_k1"
    big = dict(M=M, N=N, K=K, lddc=N)
    assert backward(g, nbytes=0, **big) == 6 and backward(g, work=NUL, **big) == 6
    need = g.gated_backward_work_size(8, 9, 64)
    assert need >= 8 * 2 * 16 * 2  # dG and dU
    assert gated_backward(g, nbytes=need - 256, dX=NUL, dW=NUL) == 0  # nothing to do
    assert gated_backward(g, nbytes=need - 1) == 6 or need % 256 == 0
    assert g.gated_backward_work_size(0, 9, 64) == 0
    # named: every part of every split; as many ways as there are steps of 64
    assert g.backward_work_size(100, 200, 300, "b128x128_k1_k1") == 0
    assert g.backward_work_size(100, 200, 300, "b128x128_k2_k1") == 4 * 2 * 100 * 300
    assert g.backward_work_size(100, 200, 300, "b256x256_k9_k2") == 4 * (4 * 100 + 2 * 200) * 300
    assert g.backward_work_size(100, 200, 300, "nope") == 0
    assert g.gated_backward_work_size(100, 200, 300, "nope") == 0
    # sums of 2^36 floats are more than a grid holds; unsplit they are none
    assert g.backward_work_size(1 << 29, 128, 128, "b256x256_k2_k1") == 0
    assert backward(g, M=1 << 29, N=128, K=128, lddc=128, lda=128, ldb=128, ldda=128, lddb=128,
                    dB=NUL, nbytes=1 << 62, config=b"b256x256_k2_k1") == 3


def test_workspaces_a_byte_too_small(g):
    """Refused by either backward call, split or not."""
    sizes = dict(M=300, K=136)
    gated_size = dict(F=200, lddh=200, ldx=136, ldw=136, ld_kept=1248, lddx=136, lddw=136)
    for config in (b"b128x128_k1_k1", b"b128x128_k2_k3", b"b256x256_k3_k2"):
        need = g.gated_backward_work_size(300, 200, 136, config.decode())
        split = 0 if config.endswith(b"k1_k1") else 4 * 136 * (
            2 * 300 + 3 * 400 if config.endswith(b"k3") else 3 * 300 + 2 * 400)
        assert need == 300 * 2 * 256 * 2 + split  # dG and dU in rows of 128-byte lines, and the parts
        assert gated_backward(g, config=config, nbytes=need - 1, **sizes, **gated_size) == 6
        need = g.backward_work_size(300, 400, 136, config.decode())
        assert need == split
        if need:
            assert backward(g, N=400, lddc=400, lda=136, ldb=136, ldda=136, lddb=136, config=config,
                            nbytes=need - 1, **sizes) == 6
    need = g.gated_backward_work_size(8, 9, 64)
    assert need == 8 * 2 * 64 * 2 and gated_backward(g, nbytes=need - 1) == 6


def test_what_is_not_used_is_not_checked(g):
    """Without dA, B may be anything, without dB A, and likewise W and X (K = 0:
    nothing is launched)."""
    assert backward(g, K=0, dA=NUL, B=ODD, ldb=3) == 0 == backward(g, K=0, dB=NUL, A=ODD, lda=3)
    assert backward(g, K=0, dA=NUL, ldb=1 << 41, ldda=1 << 41) == 0
    assert backward(g, K=0, dB=NUL, lda=1 << 41, lddb=1 << 41) == 0
    assert backward(g, K=0, dA=NUL, A=ODD) == 2 == backward(g, K=0, dB=NUL, B=ODD)
    assert backward(g, K=0, dA=NUL, lda=1 << 41) == 3 == backward(g, K=0, dB=NUL, ldda=1 << 41)
    assert gated_backward(g, K=0, dX=NUL, W=ODD, ldw=3, lddx=1 << 41) == 0
    assert gated_backward(g, K=0, dW=NUL, X=ODD, ldx=1 << 41, lddw=3) == 0
    assert gated_backward(g, K=0, dX=NUL, X=ODD) == 2 == gated_backward(g, K=0, dW=NUL, W=ODD)
    assert gated_backward(g, K=0, dX=NUL, ldx=1 << 41) == 3 == gated_backward(g, K=0, dW=NUL, ldw=1 << 41)


def test_empty_calls_launch_nothing(g):
    assert i8(g, M=0, A=NUL, SA=NUL, C=NUL) == 0 and i8(g, N=0, B=NUL, SB=NUL, C=NUL) == 0
    assert i8_gated(g, M=0, A=NUL, SA=NUL, H=NUL) == 0 and i8_gated(g, F=0, W=NUL, SW=NUL, H=NUL) == 0
    assert gated(g, M=0, X=NUL, H=NUL, kept=NUL) == 0 and gated(g, F=0, W=NUL, H=NUL) == 0
    assert quantize(g, M=0, X=NUL, Q=NUL, S=NUL) == 0
    assert backward(g, dA=NUL, dB=NUL) == 0
    assert backward(g, K=0, A=NUL, B=NUL) == 0
    assert backward(g, M=0, dC=NUL, A=NUL, dB=NUL) == 0 and backward(g, N=0, dC=NUL, B=NUL, dA=NUL) == 0
    assert gated_backward(g, dX=NUL, dW=NUL) == 0 and gated_backward(g, K=0) == 0


def test_tensor_forms_refuse_what_they_cannot_run(g):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: g.quantize_int8(x), lambda: g.matmul_int8(q, s, q, s),
                 lambda: g.gated_matmul_int8(q, s, q, s), lambda: g.gated_matmul(x, x),
                 lambda: g.matmul_backward(x[:, :4], x, x), lambda: g.gated_mlp(x, x, x[:, :2]),
                 lambda: g.gated_matmul_backward(x[:, :2], x, x, q),
                 lambda: g.gated_mlp_int8(x, q, s, q[:, :2], s)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="W1"):
        g.gated_mlp(x, x, x)


def test_gate_reference_against_differences():
    """The plain gradients that the GPU tests compare with are the plain
    gate's: central differences in 64 bits."""
    import gated_ref as ref

    rng = np.random.default_rng(0)
    g_, u, dh = rng.normal(0, 3, 500), rng.normal(0, 3, 500), rng.normal(0, 1, 500)
    s = 1e-6
    for act in ("swiglu", "geglu"):
        dg, du = ref.gate_gradients(dh, g_, u, act)
        for got, lo, hi in ((dg, ref.gate(g_ - s, u, act), ref.gate(g_ + s, u, act)),
                            (du, ref.gate(g_, u - s, act), ref.gate(g_, u + s, act))):
            # cancellation of two values of up to 50, and the third derivative
            assert np.abs(got - dh * (hi - lo) / (2 * s)).max() <= 1e-7
