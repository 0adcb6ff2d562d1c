// Launchers of the gradients' products: each grad_inst_*.hip file instantiates
// one workgroup shape of the block products' kernel for them.
#pragma once

#include "block_launch.hpp"

namespace gemm {

// op kOpBf16 or kOpF16; out kStoreF32 or that type; layout kNN or kTN.
template <int BM, int BN, int WM, int WN, int S>
hipError_t launch_grad_tile(const BlockArgs& a, int grid, hipStream_t s, int op, int out,
                            int layout) {
  auto launch = [&](auto o, auto t, auto l) {
    hipLaunchKernelGGL((block_tile_kernel<BM, BN, WM, WN, 1, S, decltype(o)::value,
                                          decltype(t)::value, kPlain, false, decltype(l)::value>),
                       dim3(grid), dim3(WM * WN * 64), 0, s, a);
    return hipGetLastError();
  };
  auto by_layout = [&](auto o, auto t) {
    return layout == kNN ? launch(o, t, std::integral_constant<int, kNN>{})
                         : launch(o, t, std::integral_constant<int, kTN>{});
  };
  const std::integral_constant<int, kStoreF32> f32{};
  if (op == kOpBf16) {
    const std::integral_constant<int, kOpBf16> o{};
    return out == kStoreF32 ? by_layout(o, f32)
                            : by_layout(o, std::integral_constant<int, kStoreBf16>{});
  }
  const std::integral_constant<int, kOpF16> o{};
  return out == kStoreF32 ? by_layout(o, f32)
                          : by_layout(o, std::integral_constant<int, kStoreF16>{});
}

// Built shapes: X(name, launcher template arguments).
#define GRAD_TILES(X)             \
  X(b256x256, 256, 256, 2, 4, 2)  \
  X(b128x128, 128, 128, 2, 2, 2)

#define GRAD_DECLARE(NAME, A, B, C, D, S)                                                 \
  extern template hipError_t launch_grad_tile<A, B, C, D, S>(const BlockArgs&, int, \
                                                             hipStream_t, int, int, int);
GRAD_TILES(GRAD_DECLARE)
#undef GRAD_DECLARE

}  // namespace gemm
