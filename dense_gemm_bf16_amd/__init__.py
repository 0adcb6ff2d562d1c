"""Python binding of ``libgemm_bf16.so``, the MI355X dense bf16 GEMM.

    C[M,N] = A[M,K] . B[N,K]^T     bf16 in, fp32 accumulate, bf16 out
                                   (gemm_f16*: the same over fp16)

and of its operators for 8-bit and mixture-of-experts layers: products over
e4m3 operands with scales per block of 128 (gemm_fp8), quantising to them
(gemm_fp8_quantize), routing (gemm_moe_route, gemm_moe_plan), the experts'
products (gemm_moe) and the weighted sum back to tokens (gemm_moe_combine);
and of dense gated layers: products over 8-bit integers (gemm_i8,
gemm_i8_quantize), gated products (gemm_gated, gemm_i8_gated) and the gradients
of dense and gated products (gemm_backward, gemm_gated_backward).

The functions here only marshal arguments (sizes, device pointers, a HIP
stream) to the C entry points of the same names declared in
``include/gemm_bf16.h``; every step of the product runs in the library's HIP
kernels.  PyTorch is used for device memory and streams only.  Importing
this package fails loudly if the library has not been built; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemm_bf16.so")

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_MISALIGNED = 2
GEMM_ERR_UNSUPPORTED = 3
GEMM_ERR_HIP = 4
GEMM_ERR_CAPTURE = 5
GEMM_ERR_SCRATCH = 6
GEMM_NOALLOC_SCRATCH_BYTES = 64 << 20
GEMM_TYPE_BF16, GEMM_TYPE_F16, GEMM_TYPE_F32, GEMM_TYPE_E4M3, GEMM_TYPE_I8 = 0, 1, 2, 3, 4
GEMM_ACT_NONE, GEMM_ACT_SWIGLU, GEMM_ACT_GEGLU = 0, 1, 2
GEMM_SCORE_SOFTMAX, GEMM_SCORE_SIGMOID = 0, 1

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with dense_gemm_bf16_amd.build.build() "
        "(hipcc, gfx950).  There is no CPU fallback.")

# PyTorch ships its own copy of the HIP runtime (same soname).  If this
# library were loaded first, the process would end up with two HIP runtimes
# (ours resolved from /opt/rocm, torch's from its own directory), and device
# pointers and streams from one would be unknown to the other.  Loading torch
# first makes the dynamic loader reuse its runtime for this library too.
try:
    import torch
except ImportError:  # plain C-ABI use without torch: /opt/rocm's runtime
    torch = None

_lib = ctypes.CDLL(LIB_PATH)
_i64, _p = ctypes.c_int64, ctypes.c_void_p
_lib.gemm_bf16.restype = ctypes.c_int
_lib.gemm_bf16.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
_lib.gemm_bf16_f32out.restype = ctypes.c_int
_lib.gemm_bf16_f32out.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
_lib.gemm_bf16_ex.restype = ctypes.c_int
_lib.gemm_bf16_ex.argtypes = [ctypes.c_char_p, _i64, _i64, _i64, _p, _i64, _p, _i64,
                              _p, _i64, ctypes.c_int, _p]
_lib.gemm_bf16_config_name.restype = ctypes.c_char_p
_lib.gemm_bf16_config_name.argtypes = [_i64, _i64, _i64]
_lib.gemm_bf16_config_at.restype = ctypes.c_char_p
_lib.gemm_bf16_config_at.argtypes = [ctypes.c_int]
_lib.gemm_bf16_status_string.restype = ctypes.c_char_p
_lib.gemm_bf16_status_string.argtypes = [ctypes.c_int]
_lib.gemm_bf16_last_hip_error.restype = ctypes.c_int
_lib.gemm_bf16_last_hip_error.argtypes = []
_lib.gemm_bf16_reserve_workspace.restype = ctypes.c_int
_lib.gemm_bf16_reserve_workspace.argtypes = [ctypes.c_size_t, _p]
_lib.gemm_bf16_workspace_size.restype = ctypes.c_size_t
_lib.gemm_bf16_workspace_size.argtypes = [_i64, _i64, _i64]
_lib.gemm_bf16_release_workspace.restype = ctypes.c_int
_lib.gemm_bf16_release_workspace.argtypes = []
_lib.gemm_f16.restype = ctypes.c_int
_lib.gemm_f16.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
_lib.gemm_f16_f32out.restype = ctypes.c_int
_lib.gemm_f16_f32out.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
_lib.gemm_f16_ex.restype = ctypes.c_int
_lib.gemm_f16_ex.argtypes = [ctypes.c_char_p, _i64, _i64, _i64, _p, _i64, _p, _i64,
                             _p, _i64, ctypes.c_int, _p]
_lib.gemm_f16_config_at.restype = ctypes.c_char_p
_lib.gemm_f16_config_at.argtypes = [ctypes.c_int]
_lib.gemm_bf16_ex_noalloc.restype = ctypes.c_int
_lib.gemm_bf16_ex_noalloc.argtypes = [ctypes.c_char_p, _i64, _i64, _i64, _p, _i64, _p, _i64,
                                      _p, _i64, ctypes.c_int, _p]
_c_int = ctypes.c_int
_fp8_args = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _c_int, _p]
_moe_args = [_c_int, _i64, _i64, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _i64, _i64,
             _p, _i64, _i64, _p, _i64, _c_int, _p]
_i8_args = [_i64, _i64, _i64, _p, _i64, _p, _p, _i64, _p, _p, _i64, _c_int, _p]
_i8_gated_args = [_i64, _i64, _i64, _p, _i64, _p, _p, _i64, _p, _c_int, _p, _i64, _c_int, _p]
_gated_args = [_c_int, _i64, _i64, _i64, _p, _i64, _p, _i64, _c_int, _p, _i64, _p, _i64, _p]
_backward_args = [_c_int, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64,
                  _c_int, _p, ctypes.c_size_t, _p]
_gated_backward_args = [_c_int, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _c_int, _p, _i64,
                        _p, _i64, _p, _i64, _c_int, _p, ctypes.c_size_t, _p]
for _name, _args in {
    "gemm_work": [_c_int, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, ctypes.c_size_t, _p],
    "gemm_backward": _backward_args,
    "gemm_backward_ex": [ctypes.c_char_p, *_backward_args],
    "gemm_gated_backward": _gated_backward_args,
    "gemm_gated_backward_ex": [ctypes.c_char_p, *_gated_backward_args],
    "gemm_i8": _i8_args,
    "gemm_i8_ex": [ctypes.c_char_p, *_i8_args],
    "gemm_i8_quantize": [_i64, _i64, _p, _i64, _c_int, _p, _i64, _p, _p],
    "gemm_i8_gated": _i8_gated_args,
    "gemm_i8_gated_ex": [ctypes.c_char_p, *_i8_gated_args],
    "gemm_gated": _gated_args,
    "gemm_gated_ex": [ctypes.c_char_p, *_gated_args],
    "gemm_fp8": _fp8_args,
    "gemm_fp8_ex": [ctypes.c_char_p, *_fp8_args],
    "gemm_fp8_quantize": [_i64, _i64, _p, _i64, _c_int, _c_int, _c_int, _p, _i64, _p, _i64, _p],
    "gemm_moe": _moe_args,
    "gemm_moe_ex": [ctypes.c_char_p, *_moe_args],
    "gemm_moe_route": [_i64, _i64, _i64, _p, _i64, _c_int, _p, _c_int, _i64, _i64, _c_int, _c_int,
                       ctypes.c_float, _p, _p, _p],
    "gemm_moe_plan": [_i64, _i64, _i64, _p, _p, _p, _p, _p],
    "gemm_moe_combine": [_i64, _i64, _i64, _i64, _p, _i64, _c_int, _p, _p, _p, _i64, _c_int, _p],
}.items():
    getattr(_lib, _name).restype = ctypes.c_int
    getattr(_lib, _name).argtypes = _args
_lib.gemm_fp8_config_name.restype = ctypes.c_char_p
_lib.gemm_fp8_config_name.argtypes = [_i64, _i64, _i64, _c_int]
_lib.gemm_moe_config_name.restype = ctypes.c_char_p
_lib.gemm_moe_config_name.argtypes = [_c_int, _i64, _i64, _i64, _i64, _c_int]
for _name in ("gemm_backward_work_size", "gemm_gated_backward_work_size"):
    getattr(_lib, _name).restype = ctypes.c_size_t
    getattr(_lib, _name).argtypes = [ctypes.c_char_p, _i64, _i64, _i64]
_lib.gemm_work_size.restype = ctypes.c_size_t
_lib.gemm_work_size.argtypes = [_c_int, _i64, _i64, _i64]
_lib.gemm_gated_kept_row.restype = ctypes.c_size_t
_lib.gemm_gated_kept_row.argtypes = [_i64]
for _name in ("gemm_backward_config_name", "gemm_gated_backward_config_name"):
    getattr(_lib, _name).restype = ctypes.c_char_p
    getattr(_lib, _name).argtypes = [_i64, _i64, _i64]
_lib.gemm_i8_config_name.restype = ctypes.c_char_p
_lib.gemm_i8_config_name.argtypes = [_i64, _i64, _i64]
_lib.gemm_i8_config_at.restype = ctypes.c_char_p
_lib.gemm_i8_config_at.argtypes = [ctypes.c_int]
_lib.gemm_gated_config_name.restype = ctypes.c_char_p
_lib.gemm_gated_config_name.argtypes = [_c_int, _i64, _i64, _i64]
_lib.gemm_fp8_config_at.restype = ctypes.c_char_p
_lib.gemm_fp8_config_at.argtypes = [ctypes.c_int]


class GemmError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        msg = status_string(status)
        if status == GEMM_ERR_HIP:
            msg += f" (hipError {last_hip_error()})"
        super().__init__(f"gemm_bf16 status {status}: {msg}")


def _ptr(x):
    """Device pointer of a torch tensor, or an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    """hipStream_t of a torch stream (default: torch's current stream)."""
    if s is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int) -> None:
    if rc != GEMM_OK:
        raise GemmError(rc)


def gemm_bf16(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C = A . B^T, bf16 output.  A, B, C: device tensors or addresses."""
    _check(_lib.gemm_bf16(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                          _stream(stream)))


def gemm_bf16_f32out(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """Same product, fp32 sums stored unrounded in C (float32)."""
    _check(_lib.gemm_bf16_f32out(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                                 _stream(stream)))


def gemm_bf16_ex(config, M, N, K, A, lda, B, ldb, C, ldc, out_f32=False,
                 stream=None) -> None:
    """As gemm_bf16 with the kernel configuration named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_bf16_ex(cfg, M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                             1 if out_f32 else 0, _stream(stream)))


def gemm_f16(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C = A . B^T over fp16 operands, fp16 output."""
    _check(_lib.gemm_f16(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                         _stream(stream)))


def gemm_f16_f32out(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """fp16 operands, fp32 sums stored unrounded in C (float32)."""
    _check(_lib.gemm_f16_f32out(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                                _stream(stream)))


def gemm_f16_ex(config, M, N, K, A, lda, B, ldb, C, ldc, out_f32=False,
                stream=None) -> None:
    """As gemm_f16 with the kernel configuration named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_f16_ex(cfg, M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                            1 if out_f32 else 0, _stream(stream)))


def gemm_bf16_ex_noalloc(config, M, N, K, A, lda, B, ldb, C, ldc, out_f32=False,
                         stream=None) -> None:
    """As gemm_bf16_ex, with the split-K partials in the library's static
    scratch array instead of an allocated workspace (nothing is allocated)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_bf16_ex_noalloc(cfg, M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                                     1 if out_f32 else 0, _stream(stream)))


def gemm_bf16_status(M, N, K, A, lda, B, ldb, C, ldc, stream=0, out_f32=False,
                     config=None, half=False) -> int:
    """Raw status code of one call (for tests of argument checking);
    ``half`` calls gemm_f16_ex instead of gemm_bf16_ex."""
    cfg = None if config is None else config.encode()
    fn = _lib.gemm_f16_ex if half else _lib.gemm_bf16_ex
    return int(fn(cfg, M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                  1 if out_f32 else 0, stream))


def config_name(M, N, K) -> str:
    return _lib.gemm_bf16_config_name(M, N, K).decode()


def config_at(i: int):
    """The i-th built configuration name, or None past the end."""
    n = _lib.gemm_bf16_config_at(i)
    return None if n is None else n.decode()


def config_names() -> list[str]:
    out = []
    while (n := config_at(len(out))) is not None:
        out.append(n)
    return out


def f16_config_at(i: int):
    """The i-th configuration built for fp16 operands, or None past the end."""
    n = _lib.gemm_f16_config_at(i)
    return None if n is None else n.decode()


def f16_config_names() -> list[str]:
    out = []
    while (n := f16_config_at(len(out))) is not None:
        out.append(n)
    return out


def status_string(status: int) -> str:
    return _lib.gemm_bf16_status_string(status).decode()


def last_hip_error() -> int:
    return int(_lib.gemm_bf16_last_hip_error())


def reserve_workspace(nbytes: int, stream=None) -> None:
    _check(_lib.gemm_bf16_reserve_workspace(nbytes, _stream(stream)))


def workspace_size(M, N, K) -> int:
    return int(_lib.gemm_bf16_workspace_size(M, N, K))


def release_workspace() -> None:
    _check(_lib.gemm_bf16_release_workspace())


# The C names, for callers who prefer them.
gemm_bf16_config_name = config_name
gemm_bf16_config_at = config_at
gemm_bf16_status_string = status_string
gemm_bf16_last_hip_error = last_hip_error
gemm_bf16_reserve_workspace = reserve_workspace
gemm_bf16_workspace_size = workspace_size
gemm_bf16_release_workspace = release_workspace
gemm_f16_config_at = f16_config_at


def _row_stride(t, rows, cols):
    """Leading dimension to pass for a 2-D tensor: its row stride, or for a
    single row (whose stride is never used) the row length rounded up to 8."""
    return t.stride(0) if rows > 1 else max(8, (cols + 7) // 8 * 8)


def matmul(A, B, out=None, out_f32=False, config=None, stream=None):
    """Convenience form on torch tensors: A (M x K, rows contiguous), B (N x K,
    rows contiguous), both bfloat16 or both float16 on the GPU; returns C
    (M x N) of the same type, or float32 with ``out_f32``."""
    import torch

    if A.dtype != B.dtype or A.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("A and B must both be torch.bfloat16 or both torch.float16")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("need A (M x K) and B (N x K)")
    if A.stride(1) != 1 or B.stride(1) != 1:
        raise ValueError("rows of A and B must be contiguous")
    M, K = A.shape
    N = B.shape[0]
    out_dtype = torch.float32 if out_f32 else A.dtype
    if out is None:
        out = torch.empty((M, N), device=A.device, dtype=out_dtype)
    if out.dtype != out_dtype or out.dim() != 2 or tuple(out.shape) != (M, N):
        raise ValueError(f"out must be a {M} x {N} {out_dtype} tensor")
    if out.stride(1) != 1:
        raise ValueError("rows of C must be contiguous")
    lda = _row_stride(A, M, K)
    ldb = _row_stride(B, N, K)
    ldc = _row_stride(out, M, N)
    fn = gemm_f16_ex if A.dtype == torch.float16 else gemm_bf16_ex
    fn(config, M, N, K, A, lda, B, ldb, out, ldc, out_f32, stream)
    return out


# ------------------------------------------------- 8-bit and mixture of experts
# The C calls, argument for argument.

def gemm_fp8(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, c_type, stream=None) -> None:
    """C = A . B^T over e4m3 operands with scales per block of 128."""
    _check(_lib.gemm_fp8(M, N, K, _ptr(A), lda, _ptr(SA), ldsa, _ptr(B), ldb, _ptr(SB), ldsb,
                         _ptr(C), ldc, c_type, _stream(stream)))


def gemm_fp8_ex(config, M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, c_type,
                stream=None) -> None:
    """As gemm_fp8 with the kernel shape named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_fp8_ex(cfg, M, N, K, _ptr(A), lda, _ptr(SA), ldsa, _ptr(B), ldb, _ptr(SB),
                            ldsb, _ptr(C), ldc, c_type, _stream(stream)))


def gemm_fp8_quantize(M, K, X, ldx, x_type, act, block_rows, Q, ldq, S, lds, stream=None) -> None:
    """X to e4m3 codes Q and scales S, per 1 x 128 or 128 x 128 block."""
    _check(_lib.gemm_fp8_quantize(M, K, _ptr(X), ldx, x_type, act, block_rows, _ptr(Q), ldq,
                                  _ptr(S), lds, _stream(stream)))


def gemm_moe(type, R, N, K, E, T, A, lda, SA, ldsa, offsets, rows, B, ldb, stride_b, SB, ldsb,
             stride_sb, C, ldc, c_type, stream=None) -> None:
    """The experts' products over rows sorted by expert."""
    gemm_moe_ex(None, type, R, N, K, E, T, A, lda, SA, ldsa, offsets, rows, B, ldb, stride_b, SB,
                ldsb, stride_sb, C, ldc, c_type, stream)


def gemm_moe_ex(config, type, R, N, K, E, T, A, lda, SA, ldsa, offsets, rows, B, ldb, stride_b, SB,
                ldsb, stride_sb, C, ldc, c_type, stream=None) -> None:
    """As gemm_moe with the kernel shape named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_moe_ex(cfg, type, R, N, K, E, T, _ptr(A), lda, _ptr(SA), ldsa, _ptr(offsets),
                            _ptr(rows), _ptr(B), ldb, stride_b, _ptr(SB), ldsb, stride_sb, _ptr(C),
                            ldc, c_type, _stream(stream)))


def gemm_moe_route(T, E, k, X, ldx, x_type, bias, score, groups, topk_groups, group_top, renorm,
                   scale, ids, weights, stream=None) -> None:
    """The top k experts of each token and their weights."""
    _check(_lib.gemm_moe_route(T, E, k, _ptr(X), ldx, x_type, _ptr(bias), score, groups,
                               topk_groups, group_top, renorm, scale, _ptr(ids), _ptr(weights),
                               _stream(stream)))


def gemm_moe_plan(T, k, E, ids, offsets, rows, pos, stream=None) -> None:
    """(token, slot) pairs sorted by expert."""
    _check(_lib.gemm_moe_plan(T, k, E, _ptr(ids), _ptr(offsets), _ptr(rows), _ptr(pos),
                              _stream(stream)))


def gemm_moe_combine(T, k, N, R, Y, ldy, y_type, pos, weights, out, ldo, out_type,
                     stream=None) -> None:
    """Each token's weighted sum of its experts' rows."""
    _check(_lib.gemm_moe_combine(T, k, N, R, _ptr(Y), ldy, y_type, _ptr(pos), _ptr(weights),
                                 _ptr(out), ldo, out_type, _stream(stream)))


def fp8_config_name(M, N, K, c_type=GEMM_TYPE_BF16) -> str:
    """The kernel shape gemm_fp8 chooses."""
    return _lib.gemm_fp8_config_name(M, N, K, c_type).decode()


def moe_config_name(type, R, N, K, E, c_type=GEMM_TYPE_BF16) -> str:
    """The kernel shape gemm_moe chooses."""
    return _lib.gemm_moe_config_name(type, R, N, K, E, c_type).decode()


def fp8_config_names() -> list[str]:
    """The kernel shapes built for gemm_fp8 and gemm_moe."""
    out = []
    while (n := _lib.gemm_fp8_config_at(len(out))) is not None:
        out.append(n.decode())
    return out


gemm_fp8_config_name = fp8_config_name
gemm_moe_config_name = moe_config_name


def gemm_fp8_config_at(i: int):
    """The i-th kernel shape of gemm_fp8 and gemm_moe, or None past the end."""
    n = _lib.gemm_fp8_config_at(i)
    return None if n is None else n.decode()


# ------------------------------------------------- 8-bit integers and gated products
# The C calls, argument for argument.

def gemm_i8(M, N, K, A, lda, SA, B, ldb, SB, C, ldc, c_type, stream=None) -> None:
    """C = A . B^T over 8-bit integers, a scale for each row of A and of B."""
    gemm_i8_ex(None, M, N, K, A, lda, SA, B, ldb, SB, C, ldc, c_type, stream)


def gemm_i8_ex(config, M, N, K, A, lda, SA, B, ldb, SB, C, ldc, c_type, stream=None) -> None:
    """As gemm_i8 with the kernel shape named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_i8_ex(cfg, M, N, K, _ptr(A), lda, _ptr(SA), _ptr(B), ldb, _ptr(SB), _ptr(C),
                           ldc, c_type, _stream(stream)))


def gemm_i8_quantize(M, K, X, ldx, x_type, Q, ldq, S, stream=None) -> None:
    """X to 8-bit integers Q with a scale for each row, S."""
    _check(_lib.gemm_i8_quantize(M, K, _ptr(X), ldx, x_type, _ptr(Q), ldq, _ptr(S),
                                 _stream(stream)))


def gemm_i8_gated(M, F, K, A, lda, SA, W, ldw, SW, act, H, ldh, h_type, stream=None) -> None:
    """H = act(A . Wg^T) * (A . Wu^T) over 8-bit integers, scaled as gemm_i8."""
    gemm_i8_gated_ex(None, M, F, K, A, lda, SA, W, ldw, SW, act, H, ldh, h_type, stream)


def gemm_i8_gated_ex(config, M, F, K, A, lda, SA, W, ldw, SW, act, H, ldh, h_type,
                     stream=None) -> None:
    """As gemm_i8_gated with the kernel shape named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_i8_gated_ex(cfg, M, F, K, _ptr(A), lda, _ptr(SA), _ptr(W), ldw, _ptr(SW), act,
                                 _ptr(H), ldh, h_type, _stream(stream)))


def gemm_gated(type, M, F, K, X, ldx, W, ldw, act, H, ldh, kept=None, ld_kept=0,
               stream=None) -> None:
    """H = act(X . Wg^T) * (X . Wu^T), bf16 or fp16; what the backward pass
    needs to `kept`."""
    gemm_gated_ex(None, type, M, F, K, X, ldx, W, ldw, act, H, ldh, kept, ld_kept, stream)


def gemm_gated_ex(config, type, M, F, K, X, ldx, W, ldw, act, H, ldh, kept=None, ld_kept=0,
                  stream=None) -> None:
    """As gemm_gated with the kernel shape named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_gated_ex(cfg, type, M, F, K, _ptr(X), ldx, _ptr(W), ldw, act, _ptr(H), ldh,
                              _ptr(kept), ld_kept, _stream(stream)))


def gemm_work(type, M, N, K, A, lda, B, ldb, C, ldc, work=None, work_bytes=0, stream=None) -> None:
    """gemm_bf16 or gemm_f16 with its workspace given."""
    _check(_lib.gemm_work(type, M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _ptr(work),
                          work_bytes, _stream(stream)))


def work_size(type, M, N, K) -> int:
    """Bytes of workspace gemm_work needs."""
    return int(_lib.gemm_work_size(type, M, N, K))


gemm_work_size = work_size


def gemm_backward(type, M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb, db_type, work=None,
                  work_bytes=0, stream=None) -> None:
    """Gradients of C = A . B^T: dA = dC . B and dB = dC^T . A."""
    gemm_backward_ex(None, type, M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb, db_type,
                     work, work_bytes, stream)


def gemm_backward_ex(config, type, M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb, db_type,
                     work=None, work_bytes=0, stream=None) -> None:
    """As gemm_backward with the plan named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_backward_ex(cfg, type, M, N, K, _ptr(dC), lddc, _ptr(A), lda, _ptr(B), ldb,
                                 _ptr(dA), ldda, _ptr(dB), lddb, db_type, _ptr(work), work_bytes,
                                 _stream(stream)))


def gemm_gated_backward(type, M, F, K, dH, lddh, X, ldx, W, ldw, act, kept, ld_kept, dX, lddx, dW,
                        lddw, dw_type, work=None, work_bytes=0, stream=None) -> None:
    """Gradients of gemm_gated's X and W from H's and what it kept."""
    gemm_gated_backward_ex(None, type, M, F, K, dH, lddh, X, ldx, W, ldw, act, kept, ld_kept, dX,
                           lddx, dW, lddw, dw_type, work, work_bytes, stream)


def gemm_gated_backward_ex(config, type, M, F, K, dH, lddh, X, ldx, W, ldw, act, kept, ld_kept, dX,
                           lddx, dW, lddw, dw_type, work=None, work_bytes=0, stream=None) -> None:
    """As gemm_gated_backward with the plan named (None = automatic)."""
    cfg = None if config is None else config.encode()
    _check(_lib.gemm_gated_backward_ex(cfg, type, M, F, K, _ptr(dH), lddh, _ptr(X), ldx, _ptr(W),
                                       ldw, act, _ptr(kept), ld_kept, _ptr(dX), lddx, _ptr(dW),
                                       lddw, dw_type, _ptr(work), work_bytes, _stream(stream)))


def backward_work_size(M, N, K, config=None) -> int:
    """Bytes of workspace gemm_backward needs (for a plan named)."""
    return int(_lib.gemm_backward_work_size(None if config is None else config.encode(), M, N, K))


def gated_backward_work_size(M, F, K, config=None) -> int:
    """Bytes of workspace gemm_gated_backward needs (for a plan named)."""
    return int(_lib.gemm_gated_backward_work_size(None if config is None else config.encode(), M, F,
                                                  K))


def backward_config_name(M, N, K) -> str:
    """The tile and the splits of K of both gradients' products."""
    return _lib.gemm_backward_config_name(M, N, K).decode()


def gated_backward_config_name(M, F, K) -> str:
    """The same of a gated product's gradients."""
    return _lib.gemm_gated_backward_config_name(M, F, K).decode()


gemm_backward_config_name = backward_config_name
gemm_gated_backward_config_name = gated_backward_config_name
gemm_backward_work_size = backward_work_size
gemm_gated_backward_work_size = gated_backward_work_size


def gated_kept_row(F) -> int:
    """Bytes that gemm_gated keeps of a row of F columns."""
    return int(_lib.gemm_gated_kept_row(F))


gemm_gated_kept_row = gated_kept_row


def i8_config_name(M, N, K) -> str:
    """The kernel shape gemm_i8 chooses."""
    return _lib.gemm_i8_config_name(M, N, K).decode()


def gated_config_name(type, M, F, K) -> str:
    """The kernel shape the gated product of a type chooses."""
    return _lib.gemm_gated_config_name(type, M, F, K).decode()


def gemm_i8_config_at(i: int):
    """The i-th kernel shape of gemm_i8 and the gated products, or None past
    the end."""
    n = _lib.gemm_i8_config_at(i)
    return None if n is None else n.decode()


def i8_config_names() -> list[str]:
    """The kernel shapes built for gemm_i8 and the gated products."""
    out = []
    while (n := gemm_i8_config_at(len(out))) is not None:
        out.append(n)
    return out


gemm_i8_config_name = i8_config_name
gemm_gated_config_name = gated_config_name


# The same on torch tensors.  These run on the tensors' device and on torch's
# current stream there; an output that is not given is allocated on it.  They
# record no gradients.

_TYPES = {} if torch is None else {
    torch.bfloat16: GEMM_TYPE_BF16, torch.float16: GEMM_TYPE_F16,
    torch.float32: GEMM_TYPE_F32, torch.float8_e4m3fn: GEMM_TYPE_E4M3}
_FLOATS = (GEMM_TYPE_BF16, GEMM_TYPE_F16, GEMM_TYPE_F32)
# torch's current device, and its current stream of a device as a hipStream_t:
# the public calls cost 0.25 and 2.8 us (the latter builds an object), these
# less than 0.1.
_raw_device = getattr(getattr(torch, "_C", None), "_cuda_getDevice", None) or (
    lambda: torch.cuda.current_device())
_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _type(t, name, allowed):
    code = _TYPES.get(t)
    if code is None or code not in allowed:
        raise TypeError(f"{name} cannot be {t}")
    return code


def _call(fn, device, *args):
    """One C call with `device` current, on torch's current stream of it."""
    index = device.index
    if index == _raw_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(index))
    if rc:
        raise GemmError(rc)


def _need(t, name, device=None, dtype=None, shape=None):
    """`t` is a tensor on the GPU (on `device`) of this type and shape, each
    of its rows contiguous."""
    if not t.is_cuda if device is None else t.device != device:
        raise ValueError(f"{name} must be on {'the GPU' if device is None else device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    # (contiguous first: the cheapest answer in the usual case)
    if not t.is_contiguous() and t.dim() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1 \
            and t.numel() > 0:
        raise ValueError(f"rows of {name} must be contiguous")


def _ld(t, unit, dim=-2):
    """Stride of a dimension, or where it is never used (one entry, empty
    rows) the row length rounded up to `unit`."""
    if t.shape[dim] > 1 and t.shape[-1] > 0:
        return t.stride(dim)
    return max(unit, -(-t.shape[-1] // unit) * unit)


def _out(out, shape, dtype, device):
    """`out` checked, or a new tensor with rows padded to 8 elements."""
    if out is None:
        # (sizes as separate arguments: 0.4 us less than as a tuple)
        rows, n = shape
        if n % 8 == 0 and n > 0:
            return torch.empty(rows, n, device=device, dtype=dtype)
        return torch.empty(rows, max(8, -(-n // 8) * 8), device=device, dtype=dtype)[:, :n]
    _need(out, "out", device, dtype, tuple(shape))
    return out


def quantize_fp8(x, act="none", block_rows=1):
    """e4m3 codes and fp32 scales of x (M x K, bfloat16, float16 or float32).

    block_rows=1: one scale for each row and 128 columns, S (ceil(K/128) x M),
    as matmul_fp8 takes for A; act="swiglu" quantises silu(g) * u, with g and u
    the two halves of x's columns.  block_rows=128: one for each 128 x 128
    block, S (ceil(M/128) x ceil(K/128)), as it takes for B.  Returns (q, S);
    q's rows are padded to 16 bytes.
    """
    _need(x, "x")
    if x.dim() != 2:
        raise ValueError("x must have two dimensions")
    if act not in ("none", "swiglu"):
        raise ValueError("act must be 'none' or 'swiglu'")
    M, K = x.shape
    if act == "swiglu":
        if K % 2:
            raise ValueError("swiglu needs an even number of columns")
        K //= 2
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    kb = -(-K // 128)
    q = torch.empty(M, max(16, -(-K // 16) * 16), device=x.device, dtype=torch.float8_e4m3fn)
    rows, cols = (kb, M) if block_rows == 1 else (-(-M // 128), kb)
    S = torch.empty(rows, cols, device=x.device, dtype=torch.float32)
    _call(_lib.gemm_fp8_quantize, x.device, M, K, x.data_ptr(), _ld(x, 1),
          _type(x.dtype, "x", _FLOATS), GEMM_ACT_SWIGLU if act == "swiglu" else GEMM_ACT_NONE,
          block_rows, q.data_ptr(), q.shape[1], S.data_ptr(), max(1, cols))
    return (q if q.shape[1] == K else q[:, :K]), S


def matmul_fp8(A, SA, B, SB, out=None, out_dtype=None, config=None):
    """C (M x N) = A . B^T of e4m3 tensors A (M x K) and B (N x K) with scales
    SA (ceil(K/128) x M) and SB (ceil(N/128) x ceil(K/128)), as quantize_fp8
    returns them.  out_dtype: bfloat16 (default), float16 or float32."""
    _need(A, "A", None, torch.float8_e4m3fn)
    dev = A.device
    _need(B, "B", dev, torch.float8_e4m3fn)
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("need A (M x K) and B (N x K)")
    (M, K), N = A.shape, B.shape[0]
    kb = -(-K // 128)
    _need(SA, "SA", dev, torch.float32, (kb, M))
    _need(SB, "SB", dev, torch.float32, (-(-N // 128), kb))
    out = _out(out, (M, N), out_dtype or (torch.bfloat16 if out is None else out.dtype), dev)
    _call(_lib.gemm_fp8_ex, dev, None if config is None else config.encode(), M, N, K,
          A.data_ptr(), _ld(A, 16), SA.data_ptr(), SA.stride(0) if kb > 1 else M, B.data_ptr(),
          _ld(B, 16), SB.data_ptr(), SB.stride(0) if N > 128 else kb, out.data_ptr(), _ld(out, 8),
          _type(out.dtype, "out", _FLOATS))
    return out


def moe_route(logits, k, bias=None, score="softmax", groups=1, topk_groups=None, group_top=2,
              renormalize=True, scale=1.0):
    """Route tokens: logits (T x E, bfloat16, float16 or float32) to
    (ids, weights), T x k each, int32 and float32.

    score "softmax" or "sigmoid"; bias (E, float32) is added to the scores for
    the choice only; a logit of -inf (or NaN) masks its expert, whatever its
    bias; of `groups` equal groups of experts the topk_groups best stay, by
    the sum of their group_top (1 or 2) best; weights are the scores of the
    chosen, divided by their sum if renormalize, times scale.  Scores that are
    equal in 64 bits go by logit, equal logits to the lowest index."""
    _need(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must have two dimensions")
    T, E = logits.shape
    dev = logits.device
    if score not in ("softmax", "sigmoid"):
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    if bias is not None:
        _need(bias, "bias", dev, torch.float32, (E,))
    ids = torch.empty(T, k, device=dev, dtype=torch.int32)
    weights = torch.empty(T, k, device=dev, dtype=torch.float32)
    _call(_lib.gemm_moe_route, dev, T, E, k, logits.data_ptr(),
          logits.stride(0) if T > 1 else E, _type(logits.dtype, "logits", _FLOATS), _ptr(bias),
          GEMM_SCORE_SIGMOID if score == "sigmoid" else GEMM_SCORE_SOFTMAX, groups,
          groups if topk_groups is None else topk_groups, group_top, 1 if renormalize else 0,
          scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def moe_plan(ids, E):
    """Sort the (token, slot) pairs of ids (T x k, int32) by expert: (offsets,
    rows, pos).  Expert e's sorted rows are offsets[e] .. offsets[e+1]-1, rows
    holds each one's token, pos (T x k) each pair's sorted row.  An id outside
    0 .. E-1 drops its pair: pos -1, and rows ends in as many -1."""
    _need(ids, "ids", None, torch.int32)
    if ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous T x k tensor")
    T, k = ids.shape
    dev = ids.device
    offsets = torch.empty(E + 1, device=dev, dtype=torch.int32)
    rows = torch.empty(T * k, device=dev, dtype=torch.int32)
    pos = torch.empty(T, k, device=dev, dtype=torch.int32)
    _call(_lib.gemm_moe_plan, dev, T, k, E, ids.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
          pos.data_ptr())
    return offsets, rows, pos


def moe_matmul(A, B, offsets, rows=None, SA=None, SB=None, out=None, out_dtype=None, config=None):
    """The experts' products: C[p] = A[rows[p]] . B[e]^T for the sorted rows p
    of each expert e, offsets[e] <= p < offsets[e+1] (A[p] without rows).

    A (T x K) and B (E x N x K): both bfloat16 or float16, or e4m3 with SA
    (ceil(K/128) x T) and SB (E x ceil(N/128) x ceil(K/128)).  C has a row for
    each entry of rows (of A without it); rows that belong to no expert are
    left as they were.  out_dtype: bfloat16, float16 or float32 (default: A's
    type, bfloat16 for e4m3)."""
    _need(A, "A")
    dev = A.device
    code = _type(A.dtype, "A", (GEMM_TYPE_BF16, GEMM_TYPE_F16, GEMM_TYPE_E4M3))
    _need(B, "B", dev, A.dtype)
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[2]:
        raise ValueError("need A (T x K) and B (E x N x K)")
    (T, K), (E, N, _) = A.shape, B.shape
    _need(offsets, "offsets", dev, torch.int32, (E + 1,))
    R = T
    if rows is not None:
        R = rows.numel()
        _need(rows, "rows", dev, torch.int32, (R,))
    scaled = code == GEMM_TYPE_E4M3
    kb, nb = -(-K // 128), -(-N // 128)
    unit = 16 if scaled else 8
    lsa = lsb = ssb = 0
    if scaled:
        if SA is None or SB is None:
            raise ValueError("e4m3 operands need SA and SB")
        _need(SA, "SA", dev, torch.float32, (kb, T))
        _need(SB, "SB", dev, torch.float32, (E, nb, kb))
        lsa = SA.stride(0) if kb > 1 else T
        lsb = SB.stride(1) if nb > 1 else kb
        ssb = SB.stride(0) if E > 1 else 0
    elif SA is not None or SB is not None:
        raise ValueError("scales go with e4m3 operands only")
    default = torch.bfloat16 if scaled else A.dtype
    out = _out(out, (R, N), out_dtype or (default if out is None else out.dtype), dev)
    _call(_lib.gemm_moe_ex, dev, None if config is None else config.encode(), code, R, N, K, E, T,
          A.data_ptr(), _ld(A, unit), _ptr(SA), lsa, offsets.data_ptr(), _ptr(rows), B.data_ptr(),
          _ld(B, unit, 1), B.stride(0) if E > 1 and K > 0 else 0, _ptr(SB), lsb, ssb, out.data_ptr(),
          _ld(out, 8), _type(out.dtype, "out", _FLOATS))
    return out


def moe_combine(Y, pos, weights, out=None, out_dtype=None):
    """out[t] = sum_j weights[t,j] Y[pos[t,j]] over the slots whose pos names a
    row of Y.  Y (R x N), pos and weights T x k; out: T x N of out_dtype
    (default Y's type)."""
    _need(Y, "Y")
    dev = Y.device
    if Y.dim() != 2 or pos.dim() != 2:
        raise ValueError("need Y (R x N), pos and weights (T x k)")
    (R, N), (T, k) = Y.shape, pos.shape
    _need(pos, "pos", dev, torch.int32)
    _need(weights, "weights", dev, torch.float32, (T, k))
    if not pos.is_contiguous() or not weights.is_contiguous():
        raise ValueError("pos and weights must be contiguous")
    y_type = _type(Y.dtype, "Y", _FLOATS)
    out = _out(out, (T, N), out_dtype or (Y.dtype if out is None else out.dtype), dev)
    _call(_lib.gemm_moe_combine, dev, T, k, N, R, Y.data_ptr(), _ld(Y, 1), y_type, pos.data_ptr(),
          weights.data_ptr(), out.data_ptr(), _ld(out, 8), _type(out.dtype, "out", _FLOATS))
    return out


def moe_mlp_fp8(x, logits, k, W1, S1, W2, S2, **route):
    """A mixture-of-experts feed-forward layer in e4m3: for each token the
    weighted sum over its k experts e of W2[e] . (silu(g) * u), (g, u) the two
    halves of W1[e] . x.

    x (T x H, bfloat16 or float16), logits (T x E); W1 (E x 2I x H) and W2
    (E x H x I) e4m3 with scales S1 (E x ceil(2I/128) x ceil(H/128)) and S2
    (E x ceil(H/128) x ceil(I/128)).  route: moe_route's keyword arguments.
    Activations are quantised per row and 128 columns before each product;
    the first product is rounded to x's type.  Returns T x H of x's type."""
    if x.dim() != 2 or logits.dim() != 2 or W1.dim() != 3:
        raise ValueError("need x (T x H), logits (T x E) and W1 (E x 2I x H)")
    # (ids past W1's experts would be dropped, and rows past x's read as zeros)
    if logits.shape[0] != x.shape[0] or logits.shape[1] != W1.shape[0]:
        raise ValueError(f"logits must have a row for each of x's {x.shape[0]} tokens and a column "
                         f"for each of W1's {W1.shape[0]} experts, not {tuple(logits.shape)}")
    if W2.shape[0] != W1.shape[0]:
        raise ValueError("W1 and W2 must hold as many experts")
    ids, weights = moe_route(logits, k, **route)
    offsets, rows, pos = moe_plan(ids, W1.shape[0])
    q, s = quantize_fp8(x)
    h = moe_matmul(q, W1, offsets, rows=rows, SA=s, SB=S1, out_dtype=x.dtype)
    q, s = quantize_fp8(h, act="swiglu")
    y = moe_matmul(q, W2, offsets, SA=s, SB=S2, out_dtype=x.dtype)
    return moe_combine(y, pos, weights)


_ACTS = {"swiglu": GEMM_ACT_SWIGLU, "geglu": GEMM_ACT_GEGLU}


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError("act must be 'swiglu' or 'geglu'")
    return code


def quantize_int8(x):
    """8-bit integers and fp32 scales of x (M x K, bfloat16, float16 or
    float32), one scale for each row: (q, S), S of M entries, as matmul_int8
    takes them for tokens and, of a weight's rows, for channels.  q's rows are
    padded to 16 bytes, from 1024 columns on to 128 (whole lines: 1 x 10240 x
    4104 16.6 -> 13.5 us, 8192 rows 328 -> 290)."""
    _need(x, "x")
    if x.dim() != 2:
        raise ValueError("x must have two dimensions")
    M, K = x.shape
    unit = 128 if K >= 1024 else 16
    q = torch.empty(M, max(16, -(-K // unit) * unit), device=x.device, dtype=torch.int8)
    S = torch.empty(M, device=x.device, dtype=torch.float32)
    _call(_lib.gemm_i8_quantize, x.device, M, K, x.data_ptr(), _ld(x, 1),
          _type(x.dtype, "x", _FLOATS), q.data_ptr(), q.shape[1], S.data_ptr())
    return (q if q.shape[1] == K else q[:, :K]), S


def _scales_of(S, name, device, n):
    _need(S, name, device, torch.float32, (n,))
    return S.data_ptr()


def matmul_int8(A, SA, B, SB, out=None, out_dtype=None, config=None):
    """C (M x N) = A . B^T of int8 tensors A (M x K) and B (N x K) with scales
    SA (M) and SB (N), as quantize_int8 returns them.  The sums are exact
    integers.  out_dtype: bfloat16 (default), float16 or float32."""
    _need(A, "A", None, torch.int8)
    dev = A.device
    _need(B, "B", dev, torch.int8)
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("need A (M x K) and B (N x K)")
    (M, K), N = A.shape, B.shape[0]
    sa, sb = _scales_of(SA, "SA", dev, M), _scales_of(SB, "SB", dev, N)
    out = _out(out, (M, N), out_dtype or (torch.bfloat16 if out is None else out.dtype), dev)
    _call(_lib.gemm_i8_ex, dev, None if config is None else config.encode(), M, N, K,
          A.data_ptr(), _ld(A, 16), sa, B.data_ptr(), _ld(B, 16), sb, out.data_ptr(), _ld(out, 8),
          _type(out.dtype, "out", _FLOATS))
    return out


def gated_matmul_int8(A, SA, W, SW, act="swiglu", out=None, out_dtype=None, config=None):
    """H (M x F) = act(A . Wg^T) * (A . Wu^T) of int8 tensors A (M x K) and W (2F
    x K: Wg's rows, then Wu's) with scales SA (M) and SW (2F).  act: "swiglu"
    (silu) or "geglu" (gelu, tanh form).  out_dtype: bfloat16 (default), float16
    or float32."""
    _need(A, "A", None, torch.int8)
    dev = A.device
    _need(W, "W", dev, torch.int8)
    if A.dim() != 2 or W.dim() != 2 or A.shape[1] != W.shape[1] or W.shape[0] % 2:
        raise ValueError("need A (M x K) and W (2F x K)")
    (M, K), F = A.shape, W.shape[0] // 2
    sa, sw = _scales_of(SA, "SA", dev, M), _scales_of(SW, "SW", dev, 2 * F)
    out = _out(out, (M, F), out_dtype or (torch.bfloat16 if out is None else out.dtype), dev)
    _call(_lib.gemm_i8_gated_ex, dev, None if config is None else config.encode(), M, F, K,
          A.data_ptr(), _ld(A, 16), sa, W.data_ptr(), _ld(W, 16), sw, _act(act), out.data_ptr(),
          _ld(out, 8), _type(out.dtype, "out", _FLOATS))
    return out


def gated_matmul(x, W, act="swiglu", out=None, save=False, config=None):
    """h (M x F) = act(g) * u with g = x . Wg^T and u = x . Wu^T: x (M x K) and W
    (2F x K: Wg's rows, then Wu's) both bfloat16 or both float16.  act: "swiglu"
    (silu) or "geglu" (gelu, tanh form).  save: return (h, kept), kept (uint8) what
    gated_matmul_backward needs: g and u to 24 bits, 6 bytes for each column.
    h is part of no autograd graph, also where x or W requires gradients."""
    _need(x, "x")
    dev, code = x.device, _type(x.dtype, "x", (GEMM_TYPE_BF16, GEMM_TYPE_F16))
    _need(W, "W", dev, x.dtype)
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1] or W.shape[0] % 2:
        raise ValueError("need x (M x K) and W (2F x K)")
    (M, K), F = x.shape, W.shape[0] // 2
    out = _out(out, (M, F), x.dtype, dev)
    kept, row = None, 0
    if save:
        row = _kept_row(F)
        kept = torch.empty(M, row, device=dev, dtype=torch.uint8)
    _call(_lib.gemm_gated_ex, dev, None if config is None else config.encode(), code, M, F, K,
          x.data_ptr(), _ld(x, 8), W.data_ptr(), _ld(W, 8), _act(act), out.data_ptr(), _ld(out, 8),
          None if kept is None else kept.data_ptr(), row)
    return (out, kept) if save else out


def _kept_row(F):
    return 6 * (-(-F // 16) * 16)


def _work(nbytes, device):
    """Workspace of one call, from torch's allocator: freed to the stream it
    was used on, and with a graph's memory while one is captured."""
    return torch.empty(nbytes, device=device, dtype=torch.uint8) if nbytes else None


def _grad(out, shape, dtype, device, name):
    """An output of a backward call: given (checked), None (new), or False
    (not wanted: None)."""
    if out is False:
        return None
    if out is None:
        return _out(None, shape, dtype, device)
    _need(out, name, device, None, shape)
    return out


def _weight_dtype(dw, dw_dtype, dtype):
    t = dw_dtype or (dtype if dw is None or dw is False else dw.dtype)
    if t not in (dtype, torch.float32):
        raise TypeError(f"a weight's gradient is {dtype} or torch.float32")
    if isinstance(dw, torch.Tensor) and dw.dtype != t:
        raise TypeError(f"the weight's gradient must be {t}")
    return t


def matmul_backward(dC, A, B, dA=None, dB=None, db_dtype=None, config=None):
    """Gradients of matmul's C = A . B^T from dC (M x N): (dA, dB) with dA = dC .
    B (M x K) and dB = dC^T . A (N x K).  dC, A and B are all bfloat16 or all
    float16.  dA, dB: tensors to write, None for new ones, False where a
    gradient is not wanted (None is returned).  db_dtype: A's type (default) or
    float32.  config: the plan's name (None = automatic)."""
    _need(dC, "dC")
    dev, dtype = dC.device, dC.dtype
    code = _type(dtype, "dC", (GEMM_TYPE_BF16, GEMM_TYPE_F16))
    if dC.dim() != 2 or A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("need dC (M x N), A (M x K) and B (N x K)")
    (M, K), N = A.shape, B.shape[0]
    _need(dC, "dC", dev, dtype, (M, N))
    _need(A, "A", dev, dtype)
    _need(B, "B", dev, dtype)
    db_dtype = _weight_dtype(dB, db_dtype, dtype)
    dA = _grad(dA, (M, K), dtype, dev, "dA")
    if dA is not None and dA.dtype != dtype:
        raise TypeError(f"dA must be {dtype}")
    dB = _grad(dB, (N, K), db_dtype, dev, "dB")
    cfg = None if config is None else config.encode()
    nbytes = _lib.gemm_backward_work_size(cfg, M, N, K)
    work = _work(nbytes, dev)
    _call(_lib.gemm_backward_ex, dev, cfg, code, M, N, K, dC.data_ptr(), _ld(dC, 8), A.data_ptr(),
          _ld(A, 8), B.data_ptr(), _ld(B, 8), _ptr(dA), 0 if dA is None else _ld(dA, 8), _ptr(dB),
          0 if dB is None else _ld(dB, 8), _TYPES[db_dtype], _ptr(work), nbytes)
    return dA, dB


def gated_matmul_backward(dh, x, W, kept, act="swiglu", dx=None, dw=None, dw_dtype=None,
                          config=None):
    """Gradients of gated_matmul's x and W from dh (M x F) and what it kept
    (save=True): (dx, dW).  act as in the forward call; dx, dw,
    dw_dtype and config as matmul_backward's dA, dB, db_dtype and config."""
    _need(x, "x")
    dev, dtype = x.device, x.dtype
    code = _type(dtype, "x", (GEMM_TYPE_BF16, GEMM_TYPE_F16))
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1] or W.shape[0] % 2:
        raise ValueError("need x (M x K) and W (2F x K)")
    (M, K), F = x.shape, W.shape[0] // 2
    _need(W, "W", dev, dtype)
    _need(dh, "dh", dev, dtype, (M, F))
    _need(kept, "kept", dev, torch.uint8, (M, _kept_row(F)))
    dw_dtype = _weight_dtype(dw, dw_dtype, dtype)
    dx = _grad(dx, (M, K), dtype, dev, "dx")
    if dx is not None and dx.dtype != dtype:
        raise TypeError(f"dx must be {dtype}")
    dw = _grad(dw, (2 * F, K), dw_dtype, dev, "dw")
    cfg = None if config is None else config.encode()
    nbytes = _lib.gemm_gated_backward_work_size(cfg, M, F, K)
    work = _work(nbytes, dev)
    _call(_lib.gemm_gated_backward_ex, dev, cfg, code, M, F, K, dh.data_ptr(), _ld(dh, 8),
          x.data_ptr(), _ld(x, 8), W.data_ptr(), _ld(W, 8), _act(act), kept.data_ptr(),
          _ld(kept, 16), _ptr(dx), 0 if dx is None else _ld(dx, 8), _ptr(dw),
          0 if dw is None else _ld(dw, 8), _TYPES[dw_dtype], _ptr(work), nbytes)
    return dx, dw


def gated_mlp(x, W1, W2, act="swiglu", save=False):
    """A gated feed-forward layer: y (M x N) = (act(g) * u) . W2^T, (g, u) the
    two halves of x . W1^T.  x (M x K), W1 (2F x K) and W2 (N x F) are all
    bfloat16 or all float16.  save: return (y, h, kept), h (M x F) and what
    gated_matmul kept, for gated_mlp_backward.  y is part of no autograd graph,
    also where x, W1 or W2 requires gradients."""
    if W2.dim() != 2 or W1.dim() != 2 or 2 * W2.shape[1] != W1.shape[0]:
        raise ValueError("need W1 (2F x K) and W2 (N x F)")
    _need(x, "x")
    dev, code = x.device, _type(x.dtype, "x", (GEMM_TYPE_BF16, GEMM_TYPE_F16))
    _need(W2, "W2", dev, x.dtype)
    r = gated_matmul(x, W1, act=act, save=save)
    h = r[0] if save else r
    (M, F), N = h.shape, W2.shape[0]
    y = _out(None, (M, N), x.dtype, dev)
    nbytes = _lib.gemm_work_size(code, M, N, F)
    work = _work(nbytes, dev)
    _call(_lib.gemm_work, dev, code, M, N, F, h.data_ptr(), _ld(h, 8), W2.data_ptr(), _ld(W2, 8),
          y.data_ptr(), _ld(y, 8), _ptr(work), nbytes)
    return (y, *r) if save else y


def gated_mlp_backward(dy, x, W1, W2, h, kept, act="swiglu", dw_dtype=None):
    """Gradients of gated_mlp from dy (M x N) and the h and kept that it returned
    with save=True: (dx, dW1, dW2), those of the weights of dw_dtype (x's type,
    the default, or float32)."""
    dh, dW2 = matmul_backward(dy, h, W2, db_dtype=dw_dtype)
    dx, dW1 = gated_matmul_backward(dh, x, W1, kept, act=act, dw_dtype=dw_dtype)
    return dx, dW1, dW2


def gated_mlp_int8(x, W1, S1, W2, S2, act="swiglu"):
    """gated_mlp over 8-bit integers: x (M x K, bfloat16 or float16), W1 (2F x K)
    and W2 (N x F) int8 with scales S1 (2F) and S2 (N), as quantize_int8 makes
    them of weights.  Activations are quantised per row before each product; h
    is rounded to x's type.  Returns M x N of x's type."""
    q, s = quantize_int8(x)
    h = gated_matmul_int8(q, s, W1, S1, act=act, out_dtype=x.dtype)
    q, s = quantize_int8(h)
    return matmul_int8(q, s, W2, S2, out_dtype=x.dtype)
