// Quantisation to 8-bit integers with one fp32 scale a row:
//
//   amax = max(largest |x| of the row, 2^-100)
//   S    = amax / 127
//   q    = x * (127 / amax), rounded to nearest even
//
// Both divisions and the product are IEEE fp32, so the codes are a function
// of the inputs alone.  |x| * (127 / amax) is at most 127 (1 + 2^-22), which
// rounds to 127.  A row that holds a NaN has a NaN scale, so that whatever it
// enters is NaN; one that holds an infinity (and no NaN) an infinite scale,
// codes of +-127 for its infinities and 0 for the rest.
#include "block_internal.h"

namespace gemm {
namespace {

constexpr float kInt8Max = 127.0f;
constexpr float kAmaxFloor = 0x1p-100f;

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 f16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef __bf16 bf16x8u __attribute__((ext_vector_type(8), aligned(2)));

template <int TYPE>
__device__ __forceinline__ float to_float(const void* p, int64_t i) {
  if constexpr (TYPE == kStoreF32) return ((const float*)p)[i];
  else if constexpr (TYPE == kStoreF16) return (float)((const _Float16*)p)[i];
  else return (float)((const __bf16*)p)[i];
}

// Elements i .. i+7, of which the first n exist (the others read 0); rows may
// start at any element.
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t i, int n, float (&v)[8]) {
  if (n >= 8) {
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

// The larger magnitude, NaN if either is one (fmaxf would drop it): of
// non-negative floats the order is that of their bits, and a NaN's are above
// infinity's.
__device__ __forceinline__ uint32_t magnitude(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
}

__device__ __forceinline__ uint32_t code(float x, float inv) {
  const float y = x * inv;
  // (an infinity of an infinite row: inf * 0)
  const float z = y != y ? __builtin_copysignf(kInt8Max, x) : y;
  return (uint32_t)(int)__builtin_rintf(z) & 0xFFu;
}

// One row a workgroup, two passes: the maximum, then the codes.
template <int TYPE>
__global__ __launch_bounds__(256) void quantize_int8_kernel(Int8QuantArgs a) {
  __shared__ uint32_t part[4];
  const int64_t m = blockIdx.x;
  const int t = threadIdx.x;
  uint32_t most = 0;
  for (int64_t k = t * 8; k < a.K; k += 256 * 8) {
    float v[8];
    load8<TYPE>(a.x, m * a.ldx + k, a.K - k < 8 ? (int)(a.K - k) : 8, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, magnitude(v[j]));
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) most = max(most, (uint32_t)__shfl_xor((int)most, d, 64));
  if ((t & 63) == 0) part[t >> 6] = most;
  __syncthreads();
  most = max(max(part[0], part[1]), max(part[2], part[3]));
  float amax = __builtin_bit_cast(float, most);
  if (amax < kAmaxFloor) amax = kAmaxFloor;  // (false for NaN)
  const float inv = kInt8Max / amax;
  if (t == 0) a.s[m] = amax / kInt8Max;
  for (int64_t k = t * 8; k < a.K; k += 256 * 8) {
    float v[8];
    const int n = a.K - k < 8 ? (int)(a.K - k) : 8;
    load8<TYPE>(a.x, m * a.ldx + k, n, v);
    u32x2 r = (u32x2){0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j >> 2] |= code(v[j], inv) << (8 * (j & 3));
    uint8_t* q = a.q + m * a.ldq + k;
    if (n == 8) {
      *(u32x2*)q = r;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = (uint8_t)(r[j >> 2] >> (8 * (j & 3)));
    }
  }
}

}  // namespace

hipError_t launch_quantize_int8(const Int8QuantArgs& a, int x_type, hipStream_t s) {
  const dim3 grid((unsigned)a.M);
  switch (x_type) {
    case kStoreBf16:
      hipLaunchKernelGGL(quantize_int8_kernel<kStoreBf16>, grid, dim3(256), 0, s, a);
      break;
    case kStoreF16:
      hipLaunchKernelGGL(quantize_int8_kernel<kStoreF16>, grid, dim3(256), 0, s, a);
      break;
    default:
      hipLaunchKernelGGL(quantize_int8_kernel<kStoreF32>, grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace gemm
