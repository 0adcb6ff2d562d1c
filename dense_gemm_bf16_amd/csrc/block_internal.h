// Host-side declarations of the 8-bit and mixture-of-experts operators: the
// kernels' launchers, shared between their files and the C entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_gemm.hpp"

namespace gemm {

// One compiled shape of the block-scaled and experts' products.  `launch`
// takes the operand type (kOp...) and the output type (kStore...).
struct BlockConfig {
  const char* name;
  int bm, bn;    // rows and columns of C per workgroup
  int threads;   // of a workgroup
  hipError_t (*launch)(const BlockArgs&, int grid, hipStream_t, int op, int out);
};

// The built shapes, terminated by an entry with name == NULL.
const BlockConfig* block_configs();

struct RouteArgs {
  const void* x;      // T rows of E logits, row stride ldx
  const float* bias;  // E, or null
  int32_t* ids;       // T x k
  float* weights;     // T x k
  int64_t T, ldx;
  int E, k, groups, topk_groups, group_top;
  bool sigmoid, renorm;
  float scale;
  int size;        // experts of a group
  float inv_size;  // 1 / size
};
hipError_t launch_route(const RouteArgs& a, int x_type, hipStream_t s);

hipError_t launch_plan(const int32_t* ids, int64_t T, int k, int E, int32_t* offsets,
                       int32_t* rows, int32_t* pos, hipStream_t s);

struct CombineArgs {
  const void* Y;       // R rows of N
  const int32_t* pos;  // T x k
  const float* w;      // T x k
  void* out;           // T rows of N
  int64_t T, N, R, ldy, ldo;
  int k;
};
hipError_t launch_combine(const CombineArgs& a, int y_type, int out_type, hipStream_t s);

struct QuantArgs {
  const void* x;
  uint8_t* q;
  float* s;
  int64_t M, K, ldx, ldq, lds;
};
hipError_t launch_quantize_rows(const QuantArgs& a, int x_type, bool swiglu, hipStream_t s);
hipError_t launch_quantize_blocks(const QuantArgs& a, int x_type, hipStream_t s);

struct Int8QuantArgs {
  const void* x;
  uint8_t* q;
  float* s;
  int64_t M, K, ldx, ldq;
};
hipError_t launch_quantize_int8(const Int8QuantArgs& a, int x_type, hipStream_t s);

struct GateGradArgs {
  const void* dH;       // M rows of F, read to F rounded up to 8
  const uint8_t* kept;  // M rows of what the forward call kept of g and u
  void* dGU;            // M rows of dg (the first Fp of ld columns) and du (of the next ld)
  int64_t M, Fp, ld, lddh, ld_kept, kept_f;
  int geglu;
};
hipError_t launch_gate_grad(const GateGradArgs& a, bool half, hipStream_t s);

// C (rows x N) = the sum of `splits` parts (rows x ld fp32, `stride` apart),
// in their order, rounded once to `out`.
struct SumParts {
  const float* parts;
  int64_t rows, ld, stride;
  int splits;  // 1 or less: nothing to do
  void* C;
  int64_t ldc, N;
  int out;
};
hipError_t launch_sum_parts(const SumParts& x, const SumParts& w, hipStream_t s);

}  // namespace gemm
