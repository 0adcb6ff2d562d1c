// Launchers of the block-scaled and experts' products: each block_inst_*.hip
// file instantiates one workgroup shape for its operand and output types.
#pragma once

#include "block_internal.h"

namespace gemm {

template <typename Launch>
hipError_t by_types(int op, int out, Launch&& launch) {
  auto by_out = [&](auto o) {
    switch (out) {
      case kStoreBf16: return launch(o, std::integral_constant<int, kStoreBf16>{});
      case kStoreF16: return launch(o, std::integral_constant<int, kStoreF16>{});
      default: return launch(o, std::integral_constant<int, kStoreF32>{});
    }
  };
  switch (op) {
    case kOpE4m3: return by_out(std::integral_constant<int, kOpE4m3>{});
    case kOpBf16: return by_out(std::integral_constant<int, kOpBf16>{});
    default: return by_out(std::integral_constant<int, kOpF16>{});
  }
}

template <int BM, int BN, int WM, int WN, int WK, int S>
hipError_t launch_block_tile(const BlockArgs& a, int grid, hipStream_t s, int op, int out) {
  return by_types(op, out, [&](auto o, auto t) {
    hipLaunchKernelGGL((block_tile_kernel<BM, BN, WM, WN, WK, S, decltype(o)::value, decltype(t)::value>),
                       dim3(grid), dim3(WM * WN * WK * 64), 0, s, a);
    return hipGetLastError();
  });
}

template <int FM, int FN, int W, int U>
hipError_t launch_block_row(const BlockArgs& a, int grid, hipStream_t s, int op, int out) {
  return by_types(op, out, [&](auto o, auto t) {
    hipLaunchKernelGGL((block_row_kernel<FM, FN, W, U, decltype(o)::value, decltype(t)::value>),
                       dim3(grid), dim3(W * 64), 0, s, a);
    return hipGetLastError();
  });
}

// Built shapes: X(name, launcher template arguments).  "k<n>": n groups of
// waves share K.
#define BLOCK_TILES(X)                \
  X(b256x256, 256, 256, 2, 4, 1, 2)   \
  X(b256x128, 256, 128, 4, 2, 1, 3)   \
  X(b128x128, 128, 128, 2, 2, 1, 2)   \
  X(b128x128k2, 128, 128, 2, 2, 2, 2) \
  X(b64x128k2, 64, 128, 2, 2, 2, 3)   \
  X(b64x64, 64, 64, 2, 2, 1, 4)       \
  X(b64x64k2, 64, 64, 2, 2, 2, 4)     \
  X(b32x128, 32, 128, 1, 4, 1, 3)     \
  X(b32x64k4, 32, 64, 2, 2, 4, 3)     \
  X(b32x32k4, 32, 32, 2, 2, 4, 4)
#define BLOCK_ROWS(X) X(r16x16, 1, 1, 8, 4)

#define BLOCK_DECLARE(NAME, A, B, C, D, E, S)                                            \
  extern template hipError_t launch_block_tile<A, B, C, D, E, S>(const BlockArgs&, int, \
                                                                 hipStream_t, int, int);
BLOCK_TILES(BLOCK_DECLARE)
#undef BLOCK_DECLARE
#define BLOCK_DECLARE(NAME, A, B, C, D)                                                      \
  extern template hipError_t launch_block_row<A, B, C, D>(const BlockArgs&, int, hipStream_t, \
                                                          int, int);
BLOCK_ROWS(BLOCK_DECLARE)
#undef BLOCK_DECLARE

}  // namespace gemm
