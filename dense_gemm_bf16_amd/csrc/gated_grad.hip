// The elementwise parts of the gradients.
//
// Of h = act(g) u with act(g) = g s(z), s the sigmoid, z = g for silu and z =
// 2 sqrt(2 / pi) (g + 0.044715 g^3) for gelu in its tanh form:
//
//   du = dh g s(z)        dg = dh u (s(z) + g s(z) s(-z) z'(g))
//
// from dh and the g and u that the forward call kept, each rounded once to the
// operands' type: they are operands of the two products that follow.  s(z) and
// s(-z) = 1 - s(z) both come from e = exp(-|z|), so neither cancels and nothing
// overflows.  Eight bytes read and four written an element: bound by memory
// (8192 x 14336: 1.4 GB in 228 us, 6.2 TB/s), for few rows by the launch (1000 x
// 1365: 5.6 us).
//
// And the sum of a split product's parts, in their order: bound by memory too
// (0.6 us a MB of parts and 3.4 for the launch).
#include "block_internal.h"

namespace gemm {
namespace {

// What a launch holds: 2^32 threads (workgroups of 256), 2^16 workgroups along
// the grid's second dimension.
constexpr int64_t kGridBlocks = (int64_t(1) << 24) - 1, kGridRows = 32768;

template <typename T>
__global__ __launch_bounds__(256) void gate_grad_kernel(GateGradArgs a) {
  typedef T t8 __attribute__((ext_vector_type(8)));
  const int64_t f = ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63)) * 8;
  if (f >= a.Fp) return;
  // (one pass but for more than 131072 rows, or 2^26 pieces of 512 columns of a
  // row: past what a grid holds, workgroups walk on)
  const int64_t step = (int64_t)gridDim.y * 4;
  for (int64_t m = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); m < a.M; m += step) {
    const t8 dh = *(const t8*)((const T*)a.dH + m * a.lddh + f);
    const uint8_t* kept = a.kept + m * a.ld_kept;
    const u32x4 gh = *(const u32x4*)(kept + f * 2), uh = *(const u32x4*)(kept + (a.kept_f + f) * 2);
    const u32x2 gl = *(const u32x2*)(kept + 4 * a.kept_f + f);
    const u32x2 ul = *(const u32x2*)(kept + 5 * a.kept_f + f);
    auto value = [](const u32x4& h, const u32x2& l, int j) {
      return kept_value(h[j >> 1] >> (16 * (j & 1)) & 0xFFFFu, l[j >> 2] >> (8 * (j & 3)) & 0xFFu);
    };
    t8 dg, du;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = (float)dh[j], g = value(gh, gl, j), u = value(uh, ul, j);
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
    T* out = (T*)a.dGU + m * 2 * a.ld + f;
    *(t8*)out = dg;
    *(t8*)(out + a.ld) = du;
  }
}

// Four columns a thread; the parts' loads do not wait for one another.
__global__ __launch_bounds__(256) void sum_parts_kernel(SumParts x, SumParts w, int first) {
  const bool is_x = (int)blockIdx.x < first;
  const SumParts& p = is_x ? x : w;
  const int64_t i = (int64_t)((int)blockIdx.x - (is_x ? 0 : first)) * 256 + threadIdx.x;
  const uint32_t quads = (uint32_t)(p.ld >> 2);
  if (i >= p.rows * quads) return;
  const float* at = p.parts + i * 4;
  f32x4 v = *(const f32x4*)at;
  int s = 1;
  for (; s + 4 <= p.splits; s += 4) {
    f32x4 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = *(const f32x4*)(at + (s + j) * p.stride);
#pragma unroll
    for (int j = 0; j < 4; ++j) v += q[j];
  }
  for (; s < p.splits; ++s) v += *(const f32x4*)(at + s * p.stride);
  const int64_t m = i / quads;
  const int n = (int)(i - m * quads) * 4;
  if (p.out == kStoreF32) store_quad<kStoreF32>(p.C, p.ldc, v, (int)m, n, (int)p.N);
  else if (p.out == kStoreF16) store_quad<kStoreF16>(p.C, p.ldc, v, (int)m, n, (int)p.N);
  else store_quad<kStoreBf16>(p.C, p.ldc, v, (int)m, n, (int)p.N);
}

int sum_blocks(const SumParts& p) { return (int)((p.rows * (p.ld >> 2) + 255) / 256); }

}  // namespace

hipError_t launch_gate_grad(const GateGradArgs& a, bool half, hipStream_t s) {
  const int64_t across = (a.Fp + 511) / 512, most = kGridBlocks / across;  // (Fp is below 2^29 + 8)
  const int64_t rows = (a.M + 3) / 4, limit = most < kGridRows ? most : kGridRows;
  const dim3 grid((unsigned)across, (unsigned)(rows < limit ? rows : limit));
  if (half)
    hipLaunchKernelGGL(gate_grad_kernel<_Float16>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(gate_grad_kernel<__bf16>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_sum_parts(const SumParts& x, const SumParts& w, hipStream_t s) {
  const int first = x.splits > 1 ? sum_blocks(x) : 0;
  const int rest = w.splits > 1 ? sum_blocks(w) : 0;
  if (first + rest == 0) return hipSuccess;
  hipLaunchKernelGGL(sum_parts_kernel, dim3((unsigned)(first + rest)), dim3(256), 0, s, x, w, first);
  return hipGetLastError();
}

}  // namespace gemm
