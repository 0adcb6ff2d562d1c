// Launchers of the gradients' products: each grad_inst_*.hip file instantiates
// one workgroup shape of the block products' kernel for them.
#pragma once

#include "block_launch.hpp"

namespace gemm {

// Both products in one launch.  op kOpBf16 or kOpF16; out_x and out_w
// kStoreF32 or that type.
struct GradPair {
  BlockArgs x, w;
  int first;     // workgroups of the first product, rounded up to a multiple of 8
  bool w_first;  // which is w's
  int grid;
};

template <int BM, int BN, int WM, int WN, int S>
hipError_t launch_grad_pair(const GradPair& p, hipStream_t s, int op, int out_x, int out_w) {
  auto launch = [&](auto o, auto tx, auto tw) {
    hipLaunchKernelGGL((grad_pair_kernel<BM, BN, WM, WN, S, decltype(o)::value,
                                         decltype(tx)::value, decltype(tw)::value>),
                       dim3(p.grid), dim3(WM * WN * 64), 0, s, p.x, p.w, p.first,
                       p.w_first ? 1 : 0);
    return hipGetLastError();
  };
  const std::integral_constant<int, kStoreF32> f32{};
  auto by_out = [&](auto o, auto own) {
    if (out_x == kStoreF32) return out_w == kStoreF32 ? launch(o, f32, f32) : launch(o, f32, own);
    return out_w == kStoreF32 ? launch(o, own, f32) : launch(o, own, own);
  };
  if (op == kOpBf16)
    return by_out(std::integral_constant<int, kOpBf16>{}, std::integral_constant<int, kStoreBf16>{});
  return by_out(std::integral_constant<int, kOpF16>{}, std::integral_constant<int, kStoreF16>{});
}

// Built shapes: X(name, launcher template arguments).
#define GRAD_TILES(X)             \
  X(b256x256, 256, 256, 2, 4, 2)  \
  X(b128x128, 128, 128, 2, 2, 2)

#define GRAD_DECLARE(NAME, A, B, C, D, S)                                                  \
  extern template hipError_t launch_grad_pair<A, B, C, D, S>(const GradPair&, hipStream_t, int, \
                                                             int, int);
GRAD_TILES(GRAD_DECLARE)
#undef GRAD_DECLARE

}  // namespace gemm
