// Gradient of h = act(g) u with act(g) = g s(z), s the sigmoid, z = g for silu
// and z = 2 sqrt(2 / pi) (g + 0.044715 g^3) for gelu in its tanh form:
//
//   du = dh g s(z)        dg = dh u (s(z) + g s(z) s(-z) z'(g))
//
// from dh and the saved g and u, each rounded once to the operands' type: they
// are operands of the two products that follow.  s(z) and s(-z) = 1 - s(z)
// both come from e = exp(-|z|), so neither cancels and nothing overflows.
//
// Elementwise, bound by memory: three values read, two written.
#include "block_internal.h"

namespace gemm {
namespace {

template <typename T>
__global__ __launch_bounds__(256) void gate_grad_kernel(GateGradArgs a) {
  typedef T t8 __attribute__((ext_vector_type(8)));
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t chunks = a.Fp >> 3;
  if (i >= a.M * chunks) return;
  const int64_t m = i / chunks, f = (i - m * chunks) * 8;
  const t8 dh = *(const t8*)((const T*)a.dH + m * a.lddh + f);
  const T* gu = (const T*)a.GU + m * a.ldgu + f;
  const t8 g8 = *(const t8*)gu, u8 = *(const t8*)(gu + a.Fp);
  t8 dg, du;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float d = (float)dh[j], g = (float)g8[j], u = (float)u8[j];
    const float z = gate_argument(g, a.geglu != 0);
    const float e = __builtin_amdgcn_exp2f(fabsf(z) * -kLog2e);
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    const float s = z >= 0.0f ? r : e * r;
    // (past 100 the second term is below fp32's smallest value; g^2 of the
    // derivative could overflow there)
    const float c = fminf(fmaxf(g, -100.0f), 100.0f);
    const float dz = a.geglu != 0 ? __builtin_fmaf(0.214064449f, c * c, 1.59576912f) : 1.0f;
    du[j] = (T)(d * (g * s));
    dg[j] = (T)(d * u * __builtin_fmaf(c * dz, e * r * r, s));
  }
  T* out = (T*)a.dGU + m * a.lddgu + f;
  *(t8*)out = dg;
  *(t8*)(out + a.Fp) = du;
}

}  // namespace

hipError_t launch_gate_grad(const GateGradArgs& a, bool half, hipStream_t s) {
  const int64_t blocks = (a.M * (a.Fp >> 3) + 255) / 256;
  if (half)
    hipLaunchKernelGGL(gate_grad_kernel<_Float16>, dim3((unsigned)blocks), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(gate_grad_kernel<__bf16>, dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace gemm
