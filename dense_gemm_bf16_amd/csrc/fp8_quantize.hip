// Quantisation to e4m3 with one fp32 scale per block:
//
//   amax = max(largest |x| of the block, 2^-100)
//   S    = amax / 448           (448: the largest e4m3 value)
//   q    = e4m3(x * (448 / amax)), rounded to nearest even
//
// in blocks of 1 x 128 (activations, optionally after silu(g) * u) or
// 128 x 128 (weights).  Both divisions and the product are IEEE fp32, so the
// codes are a function of the inputs alone.  |x| * (448 / amax) is at most
// 448 (1 + 2^-22), which rounds to 448: nothing saturates.  The floor on
// amax keeps 448 / amax finite; a block of zeros gives zeros.  The maximum
// skips NaN, which stays NaN in its own place only; a block that holds an
// infinity has an infinite scale.
//
// Bound by memory: one read of x, one write of a quarter to a half of it
// (8192 x 8192 bf16: 203 MB in 37 us, 5.5 TB/s; a copy reaches 5.0).
#include "block_internal.h"

namespace gemm {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-100f;

template <int TYPE>
__device__ __forceinline__ float to_float(const void* p, int64_t i) {
  if constexpr (TYPE == kStoreF32) return ((const float*)p)[i];
  else if constexpr (TYPE == kStoreF16) return (float)((const _Float16*)p)[i];
  else return (float)((const __bf16*)p)[i];
}

// Elements i .. i+7, of which the first n exist (the others read 0), by
// 16-byte loads where all do; rows may start at any element.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 f16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef __bf16 bf16x8u __attribute__((ext_vector_type(8), aligned(2)));

template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t i, int n, float (&v)[8]) {
  if (n == 8) {
    if constexpr (TYPE == kStoreF32) {
      const f32x4 a = *(const f32x4u*)((const float*)p + i);
      const f32x4 b = *(const f32x4u*)((const float*)p + i + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = a[j];
        v[4 + j] = b[j];
      }
    } else if constexpr (TYPE == kStoreF16) {
      const f16x8 a = *(const f16x8u*)((const _Float16*)p + i);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
    } else {
      const bf16x8 a = *(const bf16x8u*)((const __bf16*)p + i);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? to_float<TYPE>(p, i + j) : 0.0f;
  }
}

// Eight values as e4m3, packed little-endian.
__device__ __forceinline__ u32x2 pack8(const float (&v)[8], float inv) {
  u32x2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
    r[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
  }
  return r;
}

__device__ __forceinline__ void store8(uint8_t* q, int n, const u32x2& r) {
  if (n >= 8) {
    *(u32x2*)q = r;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) q[j] = (uint8_t)(r[j >> 2] >> (8 * (j & 3)));
  }
}

constexpr int kRowGroups = 32768;  // groups of four rows in the grid's second dimension

// Rows of 1 x 128 blocks.  16 lanes own one block (8 columns each), so a
// wave reads 512 columns of a row; the four waves take four rows.  (Four rows
// a wave instead, for more loads in flight: 0-68 % slower at every size from
// 64 x 2048 to 8192 x 8192.)
template <int TYPE, bool SWIGLU>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 512 + lane * 8;
  const int64_t m = ((int64_t)blockIdx.z * kRowGroups + blockIdx.y) * 4 + wave;
  if (m >= a.M) return;
  const int64_t left = a.K - col;
  const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  const int64_t at = m * a.ldx + col;
  float v[8];
  load8<TYPE>(a.x, at, n, v);
  if constexpr (SWIGLU) {
    float u[8];
    load8<TYPE>(a.x, at + a.K, n, u);  // the second half starts at column K
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] / (1.0f + expf(-v[j])) * u[j];
  }
  float amax = kAmaxFloor;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
#pragma unroll
  for (int d = 1; d < 16; d *= 2) amax = fmaxf(amax, __shfl_xor(amax, d, 64));
  if (n == 0) return;
  store8(a.q + m * a.ldq + col, n, pack8(v, kE4m3Max / amax));
  if ((lane & 15) == 0) a.s[(col >> 7) * a.lds + m] = amax / kE4m3Max;
}

// 128 x 128 blocks, one workgroup each: 16 threads a row, 8 rows a thread.
template <int TYPE>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(QuantArgs a) {
  __shared__ float wave_max[4];
  const int t = threadIdx.x;
  const int64_t col = (int64_t)blockIdx.x * 128 + (t & 15) * 8;
  const int64_t row = (int64_t)blockIdx.y * 128 + (t >> 4);
  const int64_t left = a.K - col;
  const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  float v[8][8];
  float amax = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = row + i * 16 < a.M;
    load8<TYPE>(a.x, (row + i * 16) * a.ldx + col, in ? n : 0, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) amax = fmaxf(amax, __shfl_xor(amax, d, 64));
  if ((t & 63) == 0) wave_max[t >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
  const float inv = kE4m3Max / amax;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (row + i * 16 < a.M && n > 0) store8(a.q + (row + i * 16) * a.ldq + col, n, pack8(v[i], inv));
  if (t == 0) a.s[blockIdx.y * a.lds + blockIdx.x] = amax / kE4m3Max;
}

template <int TYPE, bool SWIGLU>
hipError_t rows_of(const QuantArgs& a, hipStream_t s) {
  const int64_t groups = (a.M + 3) / 4;
  const dim3 grid((unsigned)((a.K + 511) / 512), (unsigned)(groups < kRowGroups ? groups : kRowGroups),
                  (unsigned)((groups + kRowGroups - 1) / kRowGroups));
  hipLaunchKernelGGL((quantize_rows_kernel<TYPE, SWIGLU>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantArgs& a, int x_type, bool swiglu, hipStream_t s) {
  switch (x_type) {
    case kStoreBf16: return swiglu ? rows_of<kStoreBf16, true>(a, s) : rows_of<kStoreBf16, false>(a, s);
    case kStoreF16: return swiglu ? rows_of<kStoreF16, true>(a, s) : rows_of<kStoreF16, false>(a, s);
    default: return swiglu ? rows_of<kStoreF32, true>(a, s) : rows_of<kStoreF32, false>(a, s);
  }
}

hipError_t launch_quantize_blocks(const QuantArgs& a, int x_type, hipStream_t s) {
  const dim3 grid((unsigned)((a.K + 127) / 128), (unsigned)((a.M + 127) / 128));
  switch (x_type) {
    case kStoreBf16:
      hipLaunchKernelGGL(quantize_blocks_kernel<kStoreBf16>, grid, dim3(256), 0, s, a);
      break;
    case kStoreF16:
      hipLaunchKernelGGL(quantize_blocks_kernel<kStoreF16>, grid, dim3(256), 0, s, a);
      break;
    default:
      hipLaunchKernelGGL(quantize_blocks_kernel<kStoreF32>, grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace gemm
