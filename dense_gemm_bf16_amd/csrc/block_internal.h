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

}  // namespace gemm
