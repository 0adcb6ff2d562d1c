// Launchers of the integer products and the gated products: each
// gated_inst_*.hip file instantiates workgroup shapes of the block products'
// kernels for their operand and output types.
#pragma once

#include "block_launch.hpp"

namespace gemm {

// One compiled shape.  `launch` takes the operand type (kOp...), the output
// type (kStore...), whether columns are paired, and whether B's loads are
// non-temporal; a shape that is not built for it answers hipErrorInvalidValue.
struct GatedConfig {
  const char* name;
  int bm, bn;     // rows of A and rows of B per workgroup
  int threads;    // of a workgroup
  bool gated;     // built for paired columns
  hipError_t (*launch)(const BlockArgs&, int grid, hipStream_t, int op, int out, bool gated,
                       bool stream_b);
};

// f(operand type, output type) for the types that occur: 8-bit integers with
// any output, bf16 and fp16 (gated only) with their own.
template <typename Launch>
hipError_t by_gated_types(int op, int out, bool gated, Launch&& launch) {
  typedef std::integral_constant<int, kOpI8> I8;
  auto by_mode = [&](auto o, auto t) {
    return gated ? launch(o, t, std::integral_constant<int, kGated>{})
                 : launch(o, t, std::integral_constant<int, kPlain>{});
  };
  if (op == kOpI8) {
    switch (out) {
      case kStoreBf16: return by_mode(I8{}, std::integral_constant<int, kStoreBf16>{});
      case kStoreF16: return by_mode(I8{}, std::integral_constant<int, kStoreF16>{});
      default: return by_mode(I8{}, std::integral_constant<int, kStoreF32>{});
    }
  }
  if (!gated) return hipErrorInvalidValue;
  const std::integral_constant<int, kGated> paired{};
  if (op == kOpBf16)
    return launch(std::integral_constant<int, kOpBf16>{}, std::integral_constant<int, kStoreBf16>{},
                  paired);
  return launch(std::integral_constant<int, kOpF16>{}, std::integral_constant<int, kStoreF16>{},
                paired);
}

template <int BM, int BN, int WM, int WN, int WK, int S>
hipError_t launch_gated_tile(const BlockArgs& a, int grid, hipStream_t s, int op, int out,
                             bool gated, bool stream_b) {
  return by_gated_types(op, out, gated, [&](auto o, auto t, auto m) {
    constexpr int kOp = decltype(o)::value, kOut = decltype(t)::value, kMode = decltype(m)::value;
    if constexpr (kMode == kGated && BN / WN / 16 % 2 != 0 && BM / WM / 16 % 2 != 0) {
      return hipErrorInvalidValue;  // a wave holds no whole pairs of fragments
    } else {
      const dim3 threads(WM * WN * WK * 64);
      if constexpr (BM <= 64) {
        if (stream_b) {
          hipLaunchKernelGGL((block_tile_kernel<BM, BN, WM, WN, WK, S, kOp, kOut, kMode, true>),
                             dim3(grid), threads, 0, s, a);
          return hipGetLastError();
        }
      }
      hipLaunchKernelGGL((block_tile_kernel<BM, BN, WM, WN, WK, S, kOp, kOut, kMode>), dim3(grid),
                         threads, 0, s, a);
      return hipGetLastError();
    }
  });
}

template <int FM, int FN, int W, int U, int BR>
hipError_t launch_gated_row(const BlockArgs& a, int grid, hipStream_t s, int op, int out,
                            bool gated, bool) {
  return by_gated_types(op, out, gated, [&](auto o, auto t, auto m) {
    constexpr int kMode = decltype(m)::value;
    hipLaunchKernelGGL((block_row_kernel<FM, FN, W, U, decltype(o)::value, decltype(t)::value, kMode,
                                         BR>),
                       dim3(grid), dim3(W * 64), 0, s, a);
    return hipGetLastError();
  });
}

// The block products' tiles, and one between the two largest, for products whose
// last pass over the CUs those would leave part empty (integers 777 x 10240 x
// 4104, bf16 out, 44-47 us, 256 x 256 51-54, 256 x 128 66-69; fp16 gated 777 x
// 5001 x 2055 43-44, 50, 65, each in a graph of such launches; where passes are
// whole, 6-10 % slower than 256 x 256).
#define GATED_TILES(X)               \
  BLOCK_TILES(X)                     \
  X(b256x192, 256, 192, 2, 4, 1, 2)
#define GATED_DECLARE(NAME, A, B, C, D, E, S)                                                 \
  extern template hipError_t launch_gated_tile<A, B, C, D, E, S>(const BlockArgs&, int,       \
                                                                 hipStream_t, int, int, bool, \
                                                                 bool);
GATED_TILES(GATED_DECLARE)
#undef GATED_DECLARE
// The row kernel's shapes here: X(name, fragments of A and of B, waves, steps
// ahead, rows of B in a fragment).
#define GATED_ROWS(X)          \
  X(r16x16, 1, 1, 8, 4, 16)    \
  X(r16x8, 1, 1, 8, 4, 8)      \
  X(r32x16, 2, 1, 8, 4, 16)
#define GATED_DECLARE(NAME, A, B, C, D, E)                                                     \
  extern template hipError_t launch_gated_row<A, B, C, D, E>(const BlockArgs&, int, hipStream_t, \
                                                             int, int, bool, bool);
GATED_ROWS(GATED_DECLARE)
#undef GATED_DECLARE

}  // namespace gemm
