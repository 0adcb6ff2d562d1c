// Quantisation to 8-bit integers with one fp32 scale a row:
//
//   amax = max(largest |x| of the row, 2^-100)
//   S    = amax / 127
//   q    = x * (127 * (1 / amax)), rounded to nearest even
//
// Each operation is an IEEE fp32 one, so the codes are a function of the
// inputs alone.  |x| times the factor is at most 127 (1 + 2^-21), which rounds
// to 127.  A row that holds a NaN has a NaN scale, so that whatever it
// enters is NaN; one that holds an infinity (and no NaN) an infinite scale,
// codes of +-127 for its infinities and 0 for the rest.
//
// Bound by memory: one read, one write of a quarter to a half of it (8192 x
// 8192 bf16: 201 MB in 34 us, part of the output stays in the Infinity Cache;
// a copy reaches 5.1 TB/s), and for few rows by the launch (64 x 14336: 4.1 us).
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

__device__ __forceinline__ float row_factor(uint32_t most, float* scale) {
  float amax = __builtin_bit_cast(float, most);
  if (amax < kAmaxFloor) amax = kAmaxFloor;  // (false for NaN)
  if (scale) *scale = amax / kInt8Max;
  return kInt8Max * (1.0f / amax);
}

__device__ __forceinline__ void store_codes(uint8_t* q, const float (&v)[8], float inv, int n) {
  u32x2 r = (u32x2){0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j >> 2] |= code(v[j], inv) << (8 * (j & 3));
  if (n >= 8) {
    *(u32x2*)q = r;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) q[j] = (uint8_t)(r[j >> 2] >> (8 * (j & 3)));
  }
}

// The largest magnitude over a row's WAVES waves.
template <int WAVES>
__device__ __forceinline__ uint32_t row_most(uint32_t most, uint32_t* part) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) most = max(most, (uint32_t)__shfl_xor((int)most, d, 64));
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) most = max(most, part[w]);
  }
  return most;
}

// A row in the registers of WAVES waves, NV pieces of 8 values a lane: read
// once, with all its loads in flight together.  WAVES 1: four rows a
// workgroup.
template <int TYPE, int WAVES, int NV>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void quantize_int8_kernel(
    Int8QuantArgs a) {
  __shared__ uint32_t part[WAVES];
  const int64_t m = WAVES == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (WAVES == 1 && m >= a.M) return;
  const int t = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int K = (int)a.K;
  float v[NV][8];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int k = (i * WAVES * 64 + t) * 8;
    load8<TYPE>(a.x, m * a.ldx + k, K - k < 0 ? 0 : K - k, v[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, magnitude(v[i][j]));
  const float inv = row_factor(row_most<WAVES>(most, part), t == 0 ? a.s + m : nullptr);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int k = (i * WAVES * 64 + t) * 8;
    if (k < K) store_codes(a.q + m * a.ldq + k, v[i], inv, K - k);
  }
}

// Rows of any length, two passes: the maximum, then the codes.
template <int TYPE>
__global__ __launch_bounds__(1024) void quantize_int8_long_kernel(Int8QuantArgs a) {
  __shared__ uint32_t part[16];
  const int64_t m = blockIdx.x;
  const int t = threadIdx.x;
  uint32_t most = 0;
  for (int64_t k = t * 8; k < a.K; k += 1024 * 8) {
    float v[8];
    load8<TYPE>(a.x, m * a.ldx + k, a.K - k < 8 ? (int)(a.K - k) : 8, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, magnitude(v[j]));
  }
  const float inv = row_factor(row_most<16>(most, part), t == 0 ? a.s + m : nullptr);
  for (int64_t k = t * 8; k < a.K; k += 1024 * 8) {
    float v[8];
    const int n = a.K - k < 8 ? (int)(a.K - k) : 8;
    load8<TYPE>(a.x, m * a.ldx + k, n, v);
    store_codes(a.q + m * a.ldq + k, v, inv, n);
  }
}

template <int TYPE>
hipError_t quantize(const Int8QuantArgs& a, hipStream_t s) {
  auto run = [&](auto waves, auto pieces) {
    constexpr int W = decltype(waves)::value;
    hipLaunchKernelGGL((quantize_int8_kernel<TYPE, W, decltype(pieces)::value>),
                       dim3((unsigned)(W == 1 ? (a.M + 3) / 4 : a.M)), dim3(W == 1 ? 256 : W * 64),
                       0, s, a);
    return hipGetLastError();
  };
  const std::integral_constant<int, 1> one{};
  const std::integral_constant<int, 2> two{};
  const std::integral_constant<int, 4> four{};
  const std::integral_constant<int, 16> sixteen{};
  // Short rows: a wave each.  Longer ones: four waves where rows fill the GPU
  // (8192 x 8192 34 us, sixteen waves 41; 8192 x 4096 18, 31), sixteen where
  // they do not (200 x 4096 level, 64 x 14336 4.1 us against 6.7 for four waves
  // in two passes) and past 8192 columns, where four would hold eight pieces
  // each (300 x 14336 5.8 us, four 6.9; 8192 x 14336 level).
  if (a.K <= 512) return run(one, one);
  if (a.K <= 1024) return run(one, two);
  if (a.K <= 2048) return run(one, four);
  if (a.K <= 8192 && a.M >= 256) return a.K <= 4096 ? run(four, two) : run(four, four);
  if (a.K <= 8192) return run(sixteen, one);
  if (a.K <= 16384) return run(sixteen, two);
  hipLaunchKernelGGL(quantize_int8_long_kernel<TYPE>, dim3((unsigned)a.M), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_int8(const Int8QuantArgs& a, int x_type, hipStream_t s) {
  switch (x_type) {
    case kStoreBf16: return quantize<kStoreBf16>(a, s);
    case kStoreF16: return quantize<kStoreF16>(a, s);
    default: return quantize<kStoreF32>(a, s);
  }
}

}  // namespace gemm
